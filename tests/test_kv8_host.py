"""Refusals of the query/key norm, 8-bit cache and block selection calls: on
the host, before any launch (no GPU needed)."""

import pytest
import torch

import gqa_decode_attention_place_gb300 as ga

P = 0x1000  # fake but 16-byte aligned "device" pointer: never dereferenced
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    return ga.load_library()


def test_norm_rope(lib):
    def call(q=P, k=P, qs=2048, ks=1024, wq=P, wk=P, eps=1e-6, pos=P, cos=P, sin=P, N=1, Hq=16,
             Hkv=8, D=128, L=64, qo=P, ko=P):
        return lib.attn_qk_norm_rope(q, k, qs, ks, wq, wk, eps, pos, cos, sin, N, Hq, Hkv, D, L,
                                     qo, ko, None)
    for bad in (dict(q=None), dict(k=None), dict(pos=None), dict(qo=None), dict(ko=None),
                dict(cos=None), dict(sin=None), dict(q=P + 8), dict(wq=P + 2), dict(cos=P + 4),
                dict(pos=P + 1), dict(ko=P + 8), dict(qs=2047), dict(qs=2040), dict(ks=1028),
                dict(qs=2052), dict(N=-1), dict(Hq=0), dict(Hkv=0), dict(D=0), dict(L=0),
                dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf"))):
        assert call(**bad) == INVALID, bad
    for bad in (dict(D=120), dict(D=8), dict(D=272, qs=8192, ks=8192)):
        assert call(**bad) == UNSUPPORTED, bad
    assert call(N=0, q=None, k=None) == 0


def test_norm_rope_append(lib):
    def call(q=P, k=P, v=P, qs=2048, ks=1024, vs=1024, eps=0.0, pos=P, cos=P, sin=P, kc=P, vc=P,
             B=1, S=1, Hq=16, Hkv=8, D=128, L=64, qo=P):
        return lib.attn_qk_norm_rope_append(q, k, v, qs, ks, vs, P, P, eps, pos, cos, sin, kc, vc,
                                            B, S, Hq, Hkv, D, L, qo, None)
    for bad in (dict(v=None), dict(kc=None), dict(vc=None), dict(qo=None), dict(vs=1000),
                dict(vs=1028), dict(v=P + 2), dict(kc=P + 8), dict(B=-1), dict(S=-1),
                dict(cos=None), dict(B=1 << 16, S=1 << 15)):
        assert call(**bad) == INVALID, bad
    assert call(D=40, qs=8192) == UNSUPPORTED
    assert call(S=0) == 0 and call(B=0) == 0


def test_kv8_append(lib):
    def call(kn=P, vn=P, kst=1024, vst=1024, pos=P, kc=P, vc=P, ks=P, vs=P, bounds=P, B=1, S=1,
             Hkv=8, L=64, D=128, block=64):
        return lib.attn_kv8_append(kn, vn, kst, vst, pos, kc, vc, ks, vs, bounds, B, S, Hkv, L, D,
                                   block, None)
    for bad in (dict(kn=None), dict(vn=None), dict(pos=None), dict(kc=None), dict(vc=None),
                dict(ks=None), dict(vs=None), dict(kn=P + 8), dict(bounds=P + 8), dict(ks=P + 2),
                dict(B=0), dict(S=-1), dict(Hkv=0), dict(L=0), dict(D=0), dict(block=0),
                dict(kst=1016), dict(vst=1023), dict(vst=0)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(D=64), dict(block=8), dict(block=48), dict(block=256), dict(B=8193),
                dict(Hkv=1025), dict(L=(1 << 24) + 1)):
        assert call(**bad) == UNSUPPORTED, bad
    assert call(S=0) == 0 and call(S=65) == 0  # nothing to append; no row fits


def test_kv8_decode(lib):
    need = ga.attn_kv8_workspace_size(2, 16, 8, 64, 128)
    assert need > 0 and need % 256 == 0

    def call(blocks=False, q=P, pos=P, kc=P, vc=P, ks=P, vs=P, index=P, count=4, B=2, Hq=16,
             Hkv=8, L=64, D=128, block=16, out=P, ws=P, n=need):
        if blocks:
            return lib.attn_decode_step_kv8_blocks(q, pos, kc, vc, ks, vs, index, count, B, Hq,
                                                   Hkv, L, D, block, 1.0, out, ws, n, None)
        return lib.attn_decode_step_kv8(q, pos, kc, vc, ks, vs, B, Hq, Hkv, L, D, block, 1.0, out,
                                        ws, n, None)
    for blocks in (False, True):
        for bad in (dict(q=None), dict(pos=None), dict(kc=None), dict(vs=None), dict(out=None),
                    dict(q=P + 8), dict(vc=P + 8), dict(out=P + 2), dict(ks=P + 1), dict(B=0),
                    dict(Hq=12), dict(L=0), dict(block=-16)):
            assert call(blocks, **bad) == INVALID, bad
        for bad in (dict(D=64), dict(block=24), dict(Hq=17 * 8), dict(B=8193)):
            assert call(blocks, **bad) == UNSUPPORTED, bad
        for bad in (dict(ws=None), dict(n=need - 1), dict(ws=P + 8)):
            assert call(blocks, **bad) == WORKSPACE, bad
    for bad in (dict(index=None), dict(count=0), dict(count=1 << 26), dict(index=P + 2)):
        assert call(True, **bad) == INVALID, bad


def test_scores_select_sparse(lib):
    def scores(q=P, pos=P, bounds=P, B=1, Hq=16, Hkv=8, L=64, D=128, block=16, out=P):
        return lib.attn_block_scores(q, pos, bounds, B, Hq, Hkv, L, D, block, out, None)
    for bad in (dict(q=None), dict(pos=None), dict(bounds=None), dict(out=None), dict(q=P + 4),
                dict(bounds=P + 4), dict(out=P + 2), dict(B=0), dict(Hq=9)):
        assert scores(**bad) == INVALID, bad
    for bad in (dict(D=96), dict(block=17), dict(Hq=17 * 8)):
        assert scores(**bad) == UNSUPPORTED, bad

    def select(s=P, pos=P, B=1, Hkv=8, L=64, block=16, count=3, first=1, recent=1, out=P):
        return lib.attn_block_select(s, pos, B, Hkv, L, block, count, first, recent, out, None)
    for bad in (dict(s=None), dict(pos=None), dict(out=None), dict(count=0), dict(first=-1),
                dict(recent=-1), dict(first=2, recent=2), dict(first=2 ** 31 - 1, recent=2),
                dict(L=0), dict(s=P + 2)):
        assert select(**bad) == INVALID, bad
    assert select(block=20) == UNSUPPORTED

    need = ga.attn_kv8_sparse_workspace_size(1, 16, 8, 64, 128, 16, 3)
    assert need > ga.attn_kv8_workspace_size(1, 16, 8, 64, 128)

    def sparse(q=P, pos=P, kc=P, bounds=P, count=3, first=1, recent=1, B=1, Hq=16, Hkv=8, L=64,
               D=128, block=16, out=P, ws=P, n=need):
        return lib.attn_decode_step_kv8_sparse(q, pos, kc, P, P, P, bounds, count, first, recent,
                                               B, Hq, Hkv, L, D, block, 1.0, out, ws, n, None)
    for bad in (dict(q=None), dict(pos=None), dict(kc=None), dict(bounds=None), dict(out=None),
                dict(count=0), dict(first=3, recent=1), dict(out=P + 8), dict(bounds=P + 8)):
        assert sparse(**bad) == INVALID, bad
    assert sparse(D=64) == UNSUPPORTED and sparse(block=15) == UNSUPPORTED
    assert sparse(n=need - 1) == WORKSPACE and sparse(ws=None) == WORKSPACE


def test_workspace_sizes(lib):
    size = ga.attn_kv8_workspace_size
    assert size(1, 16, 8, 64, 128) == size(1, 16, 8, 1 << 24, 128) > 0
    assert size(256, 64, 8, 8192, 128) > size(1, 64, 8, 8192, 128)
    for bad in ((0, 16, 8, 64, 128), (1, 12, 8, 64, 128), (1, 16, 8, 64, 64),
                (1, 136, 8, 64, 128), (1, 16, 8, (1 << 24) + 1, 128)):
        assert size(*bad) == 0
    assert ga.attn_kv8_sparse_workspace_size(1, 16, 8, 64, 128, 16, 0) == 0
    with pytest.raises(ga.AttnError):
        ga.kv8_workspace(1, 16, 8, 64, 64)


def test_binding_checks_tensors():
    x = torch.zeros(1, 8, 128, dtype=torch.bfloat16)
    i = torch.zeros(1, dtype=torch.int32)
    c = torch.zeros(1, 8, 16, 128, dtype=torch.uint8)
    with pytest.raises(ValueError):  # not on a GPU
        ga.attn_qk_norm_rope(x, x, None, None, 1e-6, i)
    with pytest.raises(TypeError):
        ga.attn_qk_norm_rope(x.float(), x, None, None, 1e-6, i)
    with pytest.raises(TypeError):  # codes are float8_e4m3fn tensors
        ga.attn_kv8_append(x, x, i, c, c, x, x, 16)
    with pytest.raises(TypeError):
        ga.attn_decode_step_kv8(x.float(), i, c, c, x, x, 16, 1.0)
    with pytest.raises(TypeError):
        ga.attn_block_select(x, i, 16, 16, 1)


def test_first_calls_from_several_threads():
    """The native checks are loaded once, and no thread goes on before all of it is there."""
    import threading

    from gqa_decode_attention_place_gb300 import kv8

    kv8._native = None
    kv8._address.clear()
    seen, start = [], threading.Barrier(8)

    def first():
        start.wait()
        seen.append((kv8._native or kv8._load(), len(kv8._address)))

    threads = [threading.Thread(target=first) for _ in range(8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(seen) == 8 and len({id(m) for m, _ in seen}) == 1
    assert all(n == 8 for _, n in seen)
