"""The key/value step's host side without a GPU: what the layers pass on to the calls."""
import pytest

torch = pytest.importorskip("torch")

from bitlinear_bitnet_quant_b200 import api, build_lib, chain  # noqa: E402


def _chain(**att):
    return chain.BitLinearChain([], 2, 256, 512, "cpu", attention=dict(B=2, L=1, T_cap=100, heads=2, **att))


def test_chain_passes_the_bound_on_positions(monkeypatch):
    seen = []
    monkeypatch.setattr(api, "bitnet_kv4_append", lambda *a, **kw: seen.append(("append", kw["pos"], kw["lens"])))
    monkeypatch.setattr(api, "bitnet_kv4_attention", lambda *a, **kw: seen.append(("attention", kw["pos"], kw["t_max"])))
    monkeypatch.setattr(api, "bitnet_add", lambda *a, **kw: None)
    ch = _chain(kv_bits=4)
    ch.layers = [None]
    ch.gamma_q = ch.gamma_k = [None]
    ch.kv4 = [None]
    monkeypatch.setattr(ch, "layer", lambda parts, w, stream, i: (ch.attend(i, stream), None))
    pos = torch.zeros(2, dtype=torch.int32)
    ch.forward(torch.zeros(2, 256), pos=pos, t_max=40)
    ch.forward(torch.zeros(2, 256), t0=3)
    assert seen == [("append", pos, None), ("attention", pos, 40), ("append", None, None), ("attention", None, None)]
    with pytest.raises(ValueError, match="kv_bits=4"):
        _chain().forward(torch.zeros(2, 256), t_max=10)


def test_launches_follow_the_step():
    """Per layer 8 kernels, the append and the attention's: one for few queries, two with their merge or with the
    expansion, and those again for heads that one workspace does not hold."""
    build_lib.build()
    count = api.bitnet_kv4_attention_launches
    f32, bf16 = torch.float32, torch.bfloat16
    assert count(f32, 1, 1, 2, 2, 128, 64) == 1 and count(bf16, 1, 1, 8, 2, 128, 32768) == 2
    assert count(bf16, 1, 1, 8, 2, 128, 32768, t_max=200) == 1 and count(f32, 1, 512, 16, 16, 128, 512) == 2
    assert count(f32, 1, 20, 10, 10, 128, 65536, kernel=2) == 4
    for bad in (dict(L=0), dict(B=0), dict(head_dim=32), dict(T_cap=72), dict(kernel=3), dict(t_max=65)):
        a = dict(dict(B=1, L=1, heads=2, kv_heads=2, head_dim=128, T_cap=64), **bad)
        assert count(f32, **a) == 0, bad
    make = lambda n, **att: chain.BitLinearChain([None] * n, 1, 256, 512, "cpu", attention=dict(B=1, L=1, heads=2, **att))
    assert make(3, kv_bits=4, T_cap=100).launches == make(3, T_cap=100).launches == 10 * 3 + 1
    assert make(0, kv_bits=4, T_cap=100).launches == 1
    long = make(2, kv_bits=4, T_cap=8192)
    assert long.launches == 10 * 2 + 1
    long.pos = torch.zeros(1, dtype=torch.int32)
    assert long.launches == 11 * 2 + 1
    long.t_max = 100
    assert long.launches == 10 * 2 + 1
