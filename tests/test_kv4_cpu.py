"""The key/value step without a GPU: what the entry points refuse, the cache's
packing, and the oracle's own definitions."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from bitlinear_bitnet_quant_b200 import api, build_lib  # noqa: E402
from oracle import bitnet_oracle as O  # noqa: E402
from oracle import kv4_oracle as KO  # noqa: E402

A16 = 0x10000              # fake device addresses: never dereferenced, validation fails first
BAD = 0x10008


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return api.lib()


def _rows(**kw):
    a = dict(Q=A16, K=A16, V=A16, xt=0, ldq=256, ldk=128, ldv=128, B=2, L=3, t0=0, pos=None, len=None, heads=2, kv=1,
             d=128, gq=None, gk=None, eps=1e-6, rot=128, base=1e4, flags=3, Qo=0x20000, qt=0, Kc=A16, Ks=A16, Vc=A16,
             Vs=A16, T=64)
    a.update(kw)
    return a


def _fp32(lib, **kw):
    a = _rows(**kw)
    return lib.bitnet_qk_norm_rope_append(a["Q"], a["K"], a["V"], a["xt"], a["ldq"], a["ldk"], a["ldv"], a["B"], a["L"],
                                        a["t0"], a["pos"], a["len"], a["heads"], a["kv"], a["d"], a["gq"], a["gk"],
                                        a["eps"], a["rot"], a["base"], a["Qo"], a["Kc"], a["Vc"], a["T"], None)


def _four(lib, **kw):
    a = _rows(**kw)
    return lib.bitnet_kv4_append(a["Q"], a["K"], a["V"], a["xt"], a["ldq"], a["ldk"], a["ldv"], a["B"], a["L"], a["t0"],
                               a["pos"], a["len"], a["heads"], a["kv"], a["d"], a["gq"], a["gk"], a["eps"], a["rot"],
                               a["base"], a["flags"], a["Qo"], a["qt"], a["Kc"], a["Ks"], a["Vc"], a["Vs"], a["T"],
                               None)


@pytest.mark.parametrize("call", [_fp32, _four])
def test_append_refusals(lib, call):
    assert call(lib, xt=2) == 4
    for bad in (dict(d=96), dict(heads=3, kv=2), dict(heads=0), dict(heads=257), dict(kv=0), dict(B=-1), dict(L=-1),
                dict(B=65536), dict(t0=-1), dict(t0=62), dict(T=0), dict(T=(1 << 24) + 16), dict(rot=127),
                dict(rot=130), dict(rot=-2), dict(base=1.0), dict(base=math.nan), dict(ldq=252), dict(ldk=64),
                dict(ldv=0), dict(B=1 << 15, L=1 << 15, T=1 << 24)):
        assert call(lib, **bad) == 2, bad
    assert call(lib, B=0) == 0 and call(lib, L=0) == 0
    for p in ("Q", "K", "V", "Qo", "Kc", "Vc"):
        assert call(lib, **{p: None}) == 1, p
        assert call(lib, **{p: BAD}) == 3, p
    assert call(lib, gq=BAD) == 3 and call(lib, gk=BAD) == 3
    assert call(lib, pos=A16 + 2) == 3 and call(lib, len=A16 + 2) == 3
    assert call(lib, ldq=258) == 3 and call(lib, xt=1, ldk=132) == 3          # row strides of 16 bytes
    assert call(lib, Qo=A16, ldq=512) == 2                                  # in place needs dense rows
    if call is _four:
        assert call(lib, T=72) == 2 and call(lib, flags=4) == 2 and call(lib, qt=3) == 4
        assert call(lib, Ks=None) == 1 and call(lib, Vs=BAD) == 3
        assert call(lib, Qo=A16, xt=1, ldq=256) == 2                        # in place needs one type
    else:
        assert call(lib, Qo=A16, xt=1) == 2


def test_read_and_attention_refusals(lib):
    def rd(**kw):
        a = _rows(**dict(dict(K=0x30000, V=0x40000, dt=0), **kw))
        return lib.bitnet_kv4_read(a["Kc"], a["Ks"], a["Vc"], a["Vs"], a["B"], a["L"], a["t0"], a["pos"], a["len"],
                                 a["kv"], a["d"], a["T"], a["K"], a["V"], a["dt"], None)

    def at(**kw):
        a = _rows(**dict(dict(dt=0, w=0, s=0, tm=0, A=0x30000, ws=None, wsb=0), **kw))
        return lib.bitnet_kv4_attention(a["Q"], a["dt"], a["Kc"], a["Ks"], a["Vc"], a["Vs"], a["B"], a["L"], a["t0"],
                                      a["pos"], a["len"], a["heads"], a["kv"], a["d"], a["T"], a["w"], a["s"],
                                      a["tm"], a["A"], a["ws"], a["wsb"], None)
    for call in (rd, at):
        assert call(dt=2) == 4
        for bad in (dict(d=32), dict(kv=0), dict(B=-1), dict(L=-1), dict(t0=-1), dict(t0=62), dict(T=72), dict(T=0)):
            assert call(**bad) == 2, bad
        assert call(B=0) == 0 and call(L=0) == 0
        for p in ("Kc", "Ks", "Vc", "Vs"):
            assert call(**{p: None}) == 1 and call(**{p: BAD}) == 3, p
        assert call(pos=A16 + 1) == 3
    assert rd(K=None, V=None) == 1 and rd(K=BAD) == 3
    assert at(heads=3, kv=2) == 2 and at(w=-1) == 2 and at(s=-1) == 2 and at(tm=65) == 2 and at(tm=-1) == 2
    assert at(Q=None) == 1 and at(A=None) == 1 and at(A=BAD) == 3 and at(ws=BAD) == 3
    size = lambda dt, L, T=4096, w=0, s=0, tm=0, d=128, B=2, k=0: lib.bitnet_kv4_attention_workspace_size(
        dt, B, L, 8, 2, d, T, w, s, tm, k)
    assert size(1, 1, T=512) == 0 and size(2, 512) == 0 and size(1, 512, d=32) == 0 and size(1, 512, B=0) == 0
    assert size(1, 1) == 4 * 16 * 8 * 130 * 4                             # 16 parts of 8 rows, 4 heads
    need = size(1, 2048)
    assert need == 4 * 32 * (65536 + 16)                                  # 4 heads, 32 tiles of 128 keys
    assert size(0, 2048) == 4 * 32 * (65536 + 2048)
    assert size(1, 2048, tm=3000) == 4 * 24 * (65536 + 16) and size(1, 2048, w=100, s=4) == 4 * 19 * (65536 + 16)
    assert size(1, 2048, T=1 << 24) == (1 << 17) * (65536 + 16)           # one head's share
    assert size(1, 2048, B=4096, d=64) <= 256 << 20
    assert size(1, 2048, k=1) == 0 and size(1, 1, k=2) == need and size(1, 1, k=3) == 0
    big = dict(dt=1, B=2, L=2048, heads=8, kv=2, T=4096)
    a = _rows()
    for kernel, status in ((3, 2), (-1, 2), (2, 7)):                      # no such kernels; no workspace
        assert lib.bitnet_kv4_attention_kernel(a["Q"], 0, a["Kc"], a["Ks"], a["Vc"], a["Vs"], 2, 3, 0, None, None, 2, 1,
                                               128, 64, 0, 0, 0, 0x30000, None, 0, kernel, None) == status
    assert at(**big) == 7 and at(ws=0x50000, wsb=need - 1, **big) == 7


def test_binding_refuses_host_tensors():
    q, kv = torch.zeros(2, 256), torch.zeros(2, 128)
    c = api.KV4Cache(torch.zeros(2, 1, 16, 64, dtype=torch.uint8), torch.zeros(2, 1, 16),
                     torch.zeros(2, 1, 16, 64, dtype=torch.uint8), torch.zeros(2, 1, 16))
    for call in (lambda: api.bitnet_qk_norm_rope_append(q, kv, kv, torch.zeros(2, 16, 128), torch.zeros(2, 16, 128), 2,
                                                        1, 0, 2, kv_heads=1),
                 lambda: api.bitnet_kv4_append(q, kv, kv, c, 2, 1, 0, 2),
                 lambda: api.bitnet_kv4_read(c, 2, 1, 0),
                 lambda: api.bitnet_kv4_attention(q, c, 2, 1, 0, 2)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


def test_chain_refuses_what_the_fp32_cache_lacks():
    from bitlinear_bitnet_quant_b200 import chain
    make = lambda **kw: chain.BitLinearChain([], 2, 256, 512, "cpu", attention=dict(B=2, L=1, T_cap=16, heads=2, **kw))
    for bad in (dict(kv_heads=1), dict(window=4), dict(sinks=1), dict(kv_bits=8)):
        with pytest.raises(ValueError):
            make(**bad)
    with pytest.raises(ValueError, match="kv_bits=4"):
        make().forward(torch.zeros(2, 256), pos=torch.zeros(2, dtype=torch.int32))


def test_packing():
    codes = np.array([[-8, 7, -1, 0, 1, 2, 3, -4] * 4], dtype=np.int8)
    packed = KO.pack_codes(codes)
    # word: code 2j at bits 4j, code 2j + 1 at bits 16 + 4j
    assert packed[0, :4].tolist() == [0xF8, 0x31, 0x07, 0xC2]
    assert np.array_equal(KO.unpack_codes(packed), codes)


def test_oracle_matches_the_other_definitions():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 2 * 128))
    pos = np.array([0, 1, 77, 4096, 100000])
    y = KO.turn_rows(x.reshape(5, 2, 128), pos, norm=False)
    # the two theta_i may differ by 4 roundings of 2^-53: 1e5 * 2^-51 on the largest angle, on values up to 5
    assert np.allclose(y.reshape(5, -1), O.rope_f64(x, pos, 2), rtol=0, atol=5 * 1e5 * 2.0 ** -51)
    h = KO.turn_rows(x.reshape(5, 2, 128), pos, norm=False, hadamard=True)
    assert np.allclose((h ** 2).sum(-1), (y ** 2).sum(-1))
    codes, step, _ = KO.hold_rows(y)
    top = np.abs(y).max(-1)
    assert np.abs(codes * step[..., None] - y).max() <= (top / 7).max() / 2 * 1.001 and codes.min() >= -7
    see = KO.visible(np.arange(3, 6), 6)
    assert np.array_equal(see, O.causal_mask(3, 6, 3))
    q, k, v = rng.standard_normal((3, 64)), rng.standard_normal((6, 64)), rng.standard_normal((6, 64))
    assert np.allclose(KO.attention(q, k, v, see)[0], O.attention_f64(q, k, v, 1, see))
    w = KO.visible([5], 8, window=2, sinks=1)
    assert w[0].tolist() == [True, False, False, False, True, True, False, False]
    assert not KO.attention(q, k, v, np.zeros((3, 6), bool))[0].any()
