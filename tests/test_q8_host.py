"""8-bit pools on the CPU: layout, the oracle's own codes, and the host-side
checks of the 8-bit calls (rejected before any device work)."""
import ctypes as C

import numpy as np
import pytest
import torch

import paged_kv_cache_400_b200 as pk
from oracle import quantized as oq
from paged_kv_cache_400_b200 import binding as bd

VP = C.c_void_p(16)  # never dereferenced: rejected before use


def desc(num_blocks=8, heads=2, dim=128, dtype=bd.PA_Q8_INT8, bs=16):
    return bd.pa_pool_desc(num_blocks, heads, dim, bs, dtype)


@pytest.mark.parametrize("heads,dim", [(1, 64), (3, 64), (8, 128), (32, 128), (5, 128)])
@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_pool_layout(heads, dim, code):
    p = pk.Q8Pool(3, heads, dim, code, device="cpu")
    raw = 2 * heads * 16 * dim
    assert p.buf.shape[1] % 128 == 0 and 0 <= p.buf.shape[1] - raw - 8 * heads < 128
    p.codes[1, 1, heads - 1, 15, dim - 1] = -1
    p.scales[2, 1, heads - 1] = 2.5
    assert p.buf[1, raw - 1] != 0 and int((p.buf[1] != 0).sum()) == 1
    assert p.buf[2, raw + 8 * heads - 4: raw + 8 * heads].view(torch.float32).item() == 2.5
    again = pk.Q8Pool.wrap(p.buf, heads, dim, code)
    assert torch.equal(again.scales, p.scales) and again.num_blocks == 3


def test_block_bytes_of_every_pool():
    L = bd.lib()
    assert L.pa_pool_block_bytes(desc(heads=8, dtype=bd.PA_BF16)) == 2 * 8 * 16 * 128 * 2
    assert L.pa_pool_block_bytes(desc(heads=8, dim=64, dtype=bd.PA_F32)) == 2 * 8 * 16 * 64 * 4
    assert L.pa_pool_block_bytes(desc(heads=8)) == 2 * 8 * 16 * 128 + 128
    for bad in (desc(dim=96), desc(bs=32), desc(heads=0), desc(num_blocks=0), desc(dtype=4)):
        assert L.pa_pool_block_bytes(bad) == 0


def test_wrap_refuses_other_buffers():
    n = pk.Q8Pool.block_bytes(2, 64)
    for bad in (torch.zeros(4, n + 128, dtype=torch.uint8), torch.zeros(4, n, dtype=torch.int8),
                torch.zeros(4 * n, dtype=torch.uint8), torch.zeros(8, n, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError):
            pk.Q8Pool.wrap(bad, 2, 64)
    with pytest.raises(ValueError):
        pk.Q8Pool(2, 2, 64, "int4", device="cpu")
    with pytest.raises(ValueError):
        pk.Q8Pool(2, 2, 96, device="cpu")


def test_oracle_codes_match_torch():
    """The oracle's e4m3 table and rounding against torch's conversions."""
    b = torch.arange(256, dtype=torch.uint8)
    assert np.array_equal(oq.E4M3_VALUES, b.view(torch.float8_e4m3fn).double().numpy(), equal_nan=True)
    x = torch.cat([torch.linspace(-448, 448, 20011), torch.randn(20000) * 1e-2,
                   torch.tensor([0.0, -0.0, 2.0 ** -10, 3 * 2.0 ** -10, -(2.0 ** -10), 2.0 ** -11, 447.9, 17.0, 19.0])])
    assert np.array_equal(oq.encode(x.numpy(), "e4m3"), x.to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    for code in ("int8", "e4m3"):  # every code is its own nearest code
        c = np.array([i for i in range(256) if not (code == "e4m3" and i in (127, 255) or code == "int8" and i == 128)],
                     np.uint8)
        assert np.array_equal(oq.encode(oq.decode(c, code), code), c)


def test_append_refuses_on_host():
    L = bd.lib()
    call = lambda k=VP, v=VP, pool=VP, sl=VP, n=4, d=desc(), io=bd.PA_BF16: \
        L.pa_reshape_and_cache_q8(k, v, pool, sl, n, d, io, None)
    assert call(d=desc(dtype=bd.PA_BF16)) == 2
    assert call(d=desc(dim=96)) == 2 and call(d=desc(bs=8)) == 2 and call(d=desc(heads=0)) == 1
    assert call(d=desc(heads=70000)) == 2
    assert call(io=bd.PA_Q8_INT8) == 2 and call(io=7) == 2
    assert call(n=-1) == 1
    assert call(k=None) == 1 and call(v=None) == 1 and call(pool=None) == 1 and call(sl=None) == 1
    assert call(k=C.c_void_p(24)) == 1 and call(pool=C.c_void_p(40)) == 1
    assert call(k=None, n=0) == 0


def test_plain_calls_refuse_8_bit_pools():
    L = bd.lib()
    d = desc()
    assert L.pa_reshape_and_cache(VP, VP, VP, VP, 1, d, None) == 2
    assert L.pa_decode(VP, VP, VP, VP, 4, VP, 1, 2, 0.1, d, None, 0, 16, None) == 2
    assert L.pa_prefill(VP, VP, VP, VP, 4, VP, VP, 1, 1, 2, 0.1, d, 1, None) == 2
    assert L.pa_append_decode(VP, VP, VP, VP, VP, VP, VP, 4, VP, 1, 2, 0.1, d, None, 0, 16, None) == 2
    p = pk.Q8Pool(2, 2, 64, device="cpu")
    with pytest.raises(ValueError):
        pk.pool_desc(p)


def test_binding_refuses_before_the_library():
    p = pk.Q8Pool(2, 2, 64, device="cpu")
    k = torch.zeros(3, 2, 64)
    sl = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError):  # host tensors
        pk.pa_reshape_and_cache_q8(k, k, p, sl)
    with pytest.raises(ValueError):
        pk.pa_reshape_and_cache_q8(k[:2], k, p, sl)
    with pytest.raises(ValueError):
        pk.pa_reshape_and_cache_q8(k, k, torch.zeros(2, 2, 2, 16, 64), sl)
    with pytest.raises(ValueError):
        pk.pa_copy_blocks_between(p, pk.Q8Pool(2, 2, 64, "e4m3", device="cpu"), sl.int(), sl.int())


def test_decode_refuses_on_host():
    L = bd.lib()
    call = lambda out=VP, q=VP, pool=VP, mb=4, ns=1, H=2, scale=0.1, d=desc(), io=bd.PA_BF16, ws=None, wb=0, ml=16: \
        L.pa_decode_q8(out, q, pool, VP, mb, VP, ns, H, scale, d, io, ws, wb, ml, None)
    assert call(io=bd.PA_Q8_E4M3) == 2 and call(io=-1) == 2
    assert call(d=desc(dtype=bd.PA_F32)) == 2 and call(d=desc(dim=96)) == 2 and call(d=desc(bs=32)) == 2
    assert call(H=3) == 1 and call(H=2 * 17) == 2 and call(H=0) == 1
    assert call(d=desc(heads=70000), H=70000) == 2
    assert call(ns=-1) == 1 and call(ns=70000) == 2
    assert call(ml=65) == 1 and call(ml=-1) == 1 and call(mb=0) == 1
    assert call(scale=float("inf")) == 1
    assert call(out=None) == 1 and call(q=C.c_void_p(8)) == 1
    need = L.pa_decode_q8_workspace_size(1, 2, desc(), 4096)
    assert need > 0 and L.pa_decode_q8_workspace_size(1, 2, desc(), 128) == 0
    assert call(mb=256, ml=4096) == 9 and call(mb=256, ml=4096, ws=C.c_void_p(256), wb=need - 1) == 9
    assert call(mb=256, ml=4096, ws=C.c_void_p(128), wb=need) == 1
    assert call(ns=0, out=None) == 0


def test_prefill_refuses_on_host():
    L = bd.lib()
    call = lambda out=VP, q=VP, pool=VP, mb=4, ns=2, nt=64, H=8, scale=0.1, d=desc(heads=2), mq=40: \
        L.pa_prefill_q8(out, q, pool, VP, mb, VP, VP, ns, nt, H, scale, d, mq, None)
    assert call(d=desc(dim=64)) == 2 and call(d=desc(dtype=bd.PA_BF16)) == 2
    assert call(H=6) == 2 and call(H=7) == 1 and call(H=64) == 2
    assert call(scale=-0.1) == 1 and call(scale=float("nan")) == 1
    assert call(mq=65) == 1 and call(mq=-1) == 1 and call(mb=2) == 1 and call(ns=-1) == 1 and call(ns=70000) == 2
    assert call(out=None) == 1 and call(q=C.c_void_p(8)) == 1
    assert call(ns=0, out=None) == 0 and call(mq=0, out=None) == 0
