"""The decoding operators' entry points reject bad arguments on the host, before any
launch (no GPU use), and the Python structs match the C ones."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

from block_sparse_long_04_b200 import build as _build

_build.build()
import block_sparse_long_04_b200 as xa  # noqa: E402

FAKE = 0x7F0000001000        # 16-byte aligned, never dereferenced: every call below fails first
ODD = FAKE + 2
OK, EINVAL, EUNSUP = xa.XATTN_OK, xa.XATTN_EINVAL, xa.XATTN_EUNSUPPORTED


def cache(**kw):
    a = dict(k_pages=FAKE, v_pages=FAKE, k_scale=None, v_scale=None, acc=FAKE, ordinal=FAKE,
             page_table=FAKE, lens=FAKE, B=2, Hkv=2, C=128, page=64, num_pages=10, max_pages=4, kv_type=0)
    a.update(kw)
    return bytes(xa._Cache(*[a[n] for n, _ in xa._Cache._fields_]))


def heads(H=4, data=FAKE, sb=65536, sh=8192, sm=128):
    return bytes(xa._Heads(data, sb, sh, sm, H))


def rotary(sections=(64,), axes=None, pos=FAKE, inv_freq=FAKE, pos_batch=1, interleaved=0):
    s = (ctypes.c_int * 4)(*sections)
    return bytes(xa._Rotary(pos, inv_freq, s, len(sections) if axes is None else axes, interleaved, pos_batch))


BAD_CACHES = [
    (dict(k_pages=None), EINVAL), (dict(v_pages=None), EINVAL), (dict(page_table=None), EINVAL),
    (dict(lens=None), EINVAL), (dict(k_pages=ODD), EINVAL), (dict(v_pages=ODD), EINVAL),
    (dict(acc=ODD), EINVAL), (dict(B=-1), EINVAL), (dict(Hkv=-1), EINVAL), (dict(C=0), EINVAL),
    (dict(num_pages=0), EINVAL), (dict(max_pages=0), EINVAL), (dict(kv_type=7), EINVAL),
    (dict(kv_type=1), EINVAL),                              # e4m3 without scales
    (dict(C=96), EUNSUP), (dict(page=48), EUNSUP), (dict(page=256), EUNSUP),
    (dict(max_pages=1 << 25), EUNSUP), (dict(num_pages=1 << 25), EUNSUP),
    (dict(B=65536, Hkv=1), EUNSUP), (dict(B=40000, Hkv=2), EUNSUP),
]


def test_structs_match_the_header(tmp_path, repo_root):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("needs a C compiler")
    names = {"xattn_heads": xa._Heads, "xattn_rotary": xa._Rotary, "xattn_cache": xa._Cache}
    lines = []
    for c, py in names.items():
        lines.append(f'printf("%zu\\n", sizeof({c}));')
        lines += [f'printf("%zu\\n", offsetof({c}, {f}));' for f, _ in py._fields_]
    src = tmp_path / "s.c"
    src.write_text('#include "xattn.h"\n#include <stdio.h>\nint main(void) {' + "".join(lines) + "return 0;}")
    exe = tmp_path / "s"
    subprocess.check_call([gcc, "-I", os.path.join(repo_root, "include"), str(src), "-o", str(exe)])
    got = [int(x) for x in subprocess.check_output([str(exe)]).split()]
    want = []
    for py in names.values():
        want.append(ctypes.sizeof(py))
        want += [getattr(py, f).offset for f, _ in py._fields_]
    assert got == want
    # and the packers write that layout
    assert xa._pack_heads(1, 2, 3, 4, 5) == bytes(xa._Heads(1, 2, 3, 4, 5))
    assert xa._pack_rotary(1, 2, 3, 4, 5, 6, 7, True, 9) == \
        bytes(xa._Rotary(1, 2, (ctypes.c_int * 4)(3, 4, 5, 6), 7, 1, 9))
    assert xa._pack_cache(*range(15)) == bytes(xa._Cache(*range(15)))


# ------------------------------------------------------------------- rope
def _rope(Q=None, K=None, rot=None, inverse=0, B=2, M=64, C=128, Qo=None, Ko=None, null=()):
    a = dict(Q=Q or heads(4), K=K or heads(2), rot=rot or rotary(), Qo=Qo or heads(4), Ko=Ko or heads(2))
    for n in null:
        a[n] = None
    return xa._lib.xattn_rope(a["Q"], a["K"], a["rot"], inverse, B, M, C, a["Qo"], a["Ko"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(B=-1), EINVAL), (dict(M=-1), EINVAL), (dict(C=0), EINVAL), (dict(C=96), EUNSUP),
    (dict(B=65536), EUNSUP),
    (dict(rot=rotary((0,))), EINVAL), (dict(rot=rotary((72,))), EINVAL), (dict(rot=rotary((32, -8))), EINVAL),
    (dict(rot=rotary((12,))), EUNSUP), (dict(rot=rotary((20, 20, 20))), EUNSUP),
    (dict(rot=rotary((64,), axes=0)), EINVAL), (dict(rot=rotary((64,), axes=5)), EINVAL),
    (dict(rot=rotary(pos=None)), EINVAL), (dict(rot=rotary(inv_freq=None)), EINVAL),
    (dict(rot=rotary(pos_batch=3)), EINVAL), (dict(null=("rot",)), EINVAL),
    (dict(null=("Q",)), EINVAL), (dict(null=("Qo",)), EINVAL), (dict(null=("K",)), EINVAL),
    (dict(null=("Ko",)), EINVAL), (dict(Qo=heads(3)), EINVAL), (dict(Ko=heads(4)), EINVAL),
    (dict(Q=heads(4, data=None)), EINVAL), (dict(Q=heads(4, data=ODD)), EINVAL),
    (dict(Qo=heads(4, data=ODD)), EINVAL), (dict(Q=heads(-1)), EINVAL),
    (dict(Q=heads(4, sm=100)), EUNSUP), (dict(K=heads(2, sh=8196)), EUNSUP),
    (dict(Qo=heads(4, sh=0)), EINVAL), (dict(Qo=heads(4, sm=0)), EINVAL), (dict(Qo=heads(4, sb=0)), EINVAL),
    (dict(B=0), OK), (dict(M=0), OK), (dict(Q=heads(0), Qo=heads(0), K=heads(0), Ko=heads(0)), OK),
    (dict(Q=heads(0), Qo=heads(0), null=("K", "Ko")), OK),
])
def test_rope_rejects_on_host(kw, want):
    assert _rope(**kw) == want


# ----------------------------------------------------------------- append
def _append(c=None, K=None, V=None, T=8, rope=False, rot=None, Q=None, Qo=None):
    K, V = K or heads(2), V or heads(2)
    c = cache() if c is None else c
    if rope:
        return xa._lib.xattn_rope_append(Q or heads(4), K, V, rot or rotary(), c, T, None, None,
                                         Qo or heads(4), None)
    return xa._lib.xattn_cache_append(K, V, c, T, None, None, None)


@pytest.mark.parametrize("rope", [False, True])
@pytest.mark.parametrize("kw,want", BAD_CACHES)
def test_append_rejects_bad_caches(kw, want, rope):
    assert _append(cache(**kw), rope=rope) == want


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), EINVAL), (dict(K=heads(3)), EINVAL), (dict(V=heads(1)), EINVAL),
    (dict(K=heads(2, data=None)), EINVAL), (dict(V=heads(2, data=ODD)), EINVAL),
    (dict(V=heads(2, sm=4)), EUNSUP),
    (dict(rope=True, rot=rotary((72,))), EINVAL), (dict(rope=True, rot=rotary((12,))), EUNSUP),
    (dict(rope=True, rot=rotary(pos_batch=3)), EINVAL), (dict(rope=True, Qo=heads(2)), EINVAL),
    (dict(rope=True, Q=heads(4, data=ODD)), EINVAL), (dict(rope=True, Qo=heads(4, sh=0)), EINVAL),
    (dict(T=0), OK), (dict(T=0, rope=True), OK),
    (dict(c=cache(B=0)), OK), (dict(c=cache(Hkv=0), K=heads(0), V=heads(0)), OK),
])
def test_append_rejects_on_host(kw, want):
    assert _append(**kw) == want


def test_append_needs_its_structs():
    assert xa._lib.xattn_cache_append(None, heads(2), cache(), 8, None, None, None) == EINVAL
    assert xa._lib.xattn_cache_append(heads(2), None, cache(), 8, None, None, None) == EINVAL
    assert xa._lib.xattn_cache_append(heads(2), heads(2), None, 8, None, None, None) == EINVAL
    assert xa._lib.xattn_rope_append(heads(4), heads(2), heads(2), None, cache(), 8, None, None,
                                     heads(4), None) == EINVAL


# ----------------------------------------------------------------- decode
def _decode(c=None, Q=None, scale=0.1, O=FAKE, lse=None, acc_out=None, ws=FAKE, ws_bytes=1 << 40):
    return xa._lib.xattn_decode_attn(Q or heads(4), cache() if c is None else c, scale, O, lse, acc_out,
                                     ws, ws_bytes, None)


@pytest.mark.parametrize("kw,want", BAD_CACHES)
def test_decode_rejects_bad_caches(kw, want):
    assert _decode(cache(**kw)) == want
    assert xa._lib.xattn_decode_workspace_size(cache(**kw), 4, 0) == 0


@pytest.mark.parametrize("kw,want", [
    (dict(Q=heads(3)), EINVAL), (dict(Q=heads(-2)), EINVAL), (dict(Q=heads(258)), EUNSUP),
    (dict(Q=heads(4, data=None)), EINVAL), (dict(Q=heads(4, data=ODD)), EINVAL),
    (dict(Q=heads(4, sh=4)), EUNSUP), (dict(scale=0.0), EINVAL), (dict(scale=-1.0), EINVAL),
    (dict(scale=float("nan")), EINVAL), (dict(scale=float("inf")), EINVAL),
    (dict(O=None), EINVAL), (dict(O=ODD), EINVAL), (dict(ws=None), EINVAL), (dict(ws=ODD), EINVAL),
    (dict(ws_bytes=64), EINVAL), (dict(c=cache(acc=None), acc_out=FAKE), EINVAL),
    (dict(c=cache(Hkv=0)), EINVAL),
    (dict(c=cache(B=0)), OK), (dict(Q=heads(0)), OK), (dict(c=cache(Hkv=0), Q=heads(0)), OK),
])
def test_decode_rejects_on_host(kw, want):
    assert _decode(**kw) == want


def test_decode_workspace_size():
    size = xa._lib.xattn_decode_workspace_size
    assert size(cache(), 4, 0) > 0
    # the weights add one fp32 logit per query head and slot
    assert size(cache(), 4, 1) - size(cache(), 4, 0) == 2 * 4 * 4 * 64 * 4
    assert _decode(acc_out=FAKE, ws_bytes=size(cache(), 4, 1) - 1) == EINVAL
    assert _decode(ws_bytes=size(cache(), 4, 0) - 1) == EINVAL
    assert size(cache(B=0), 4, 0) == 0 and size(None, 4, 0) == 0 and size(cache(), 3, 0) == 0


@pytest.mark.parametrize("kw,want", [
    (dict(), EINVAL),                                            # a workspace of no bytes
    (dict(Q=heads(3)), EINVAL), (dict(Q=heads(258)), EUNSUP), (dict(c=cache(page=48)), EUNSUP),
    (dict(acc_out=FAKE + 4), EINVAL), (dict(c=cache(acc=None), acc_out=FAKE), EINVAL), (dict(scale=-1.0), EINVAL),
    (dict(c=cache(B=0)), OK), (dict(Q=heads(0)), OK),
])
def test_decode_with_idle_sequences_rejects_on_host(kw, want):
    a = dict(c=cache(), Q=heads(4), scale=0.1, acc_out=None)
    a.update(kw)
    for n_new in (None, FAKE):
        assert xa._lib.xattn_decode_attn_ex(a["Q"], a["c"], n_new, a["scale"], FAKE, None, a["acc_out"], FAKE, 0,
                                            None) == want

@pytest.mark.parametrize("off", [4, 8, 12])
def test_decode_rejects_an_unaligned_acc_out(off):
    """acc_out is stored 16 bytes at a time, like the cache's own acc."""
    assert _decode(acc_out=FAKE + off) == EINVAL


@pytest.mark.parametrize("scale", [2.5e38, 3.4e38])
def test_decode_rejects_a_scale_that_overflows_in_log2_units(scale):
    assert _decode(scale=scale) == EINVAL


# ------------------------------------------------------------------ evict
def _evict(c=None, budget=100, recent=8, sink=4, acc_out=FAKE, ord_out=FAKE, ws=FAKE, ws_bytes=1 << 40):
    return xa._lib.xattn_cache_evict(cache() if c is None else c, budget, recent, sink, None, acc_out,
                                     ord_out, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,want", BAD_CACHES)
def test_evict_rejects_bad_caches(kw, want):
    assert _evict(cache(**kw)) == want
    assert xa._lib.xattn_cache_evict_workspace_size(cache(**kw), 100) == 0


@pytest.mark.parametrize("kw,want", [
    (dict(budget=0), EINVAL), (dict(budget=-3), EINVAL), (dict(recent=-1), EINVAL), (dict(sink=-1), EINVAL),
    (dict(recent=97, sink=4), EINVAL), (dict(budget=1 << 20, recent=(1 << 31) - 1, sink=(1 << 31) - 1), EINVAL),
    (dict(acc_out=None), EINVAL), (dict(ord_out=None), EINVAL), (dict(ws=None), EINVAL), (dict(ws=ODD), EINVAL),
    (dict(acc_out=ODD), EINVAL), (dict(ord_out=ODD), EINVAL), (dict(ws_bytes=8), EINVAL),
    (dict(c=cache(acc=None)), EINVAL), (dict(c=cache(ordinal=None)), EINVAL), (dict(c=cache(B=0)), OK),
])
def test_evict_rejects_on_host(kw, want):
    assert _evict(**kw) == want


def test_evict_workspace_size():
    size = xa._lib.xattn_cache_evict_workspace_size
    # at most min(budget, capacity - budget) moves of a row, two lists, and the counts
    assert size(cache(), 100) == 256 + 2 * ((4 * 100 * 4 + 255) // 256 * 256)
    assert size(cache(), 200) == 256 + 2 * ((4 * 56 * 4 + 255) // 256 * 256)
    assert size(cache(), 256) == 256 and size(cache(), 10000) == 256
    assert size(cache(), 0) == 0 and size(None, 5) == 0


def _evict_plan(B, Hkv, page, max_pages, budget):
    """(rows, CTAs per row, most slots of one, bytes ahead of the keys) as the library plans them."""
    def up(x):
        return (x + 255) // 256 * 256

    cap, rows, cluster = max_pages * page, B * Hkv, 1
    while cluster < 8 and rows * cluster * 2 <= 148 and cap // (cluster * 2) >= 2048:
        cluster *= 2
    share = (-(-cap // cluster) + 3) // 4 * 4
    moves = max(0, min(budget, cap - budget))
    return rows, cluster, share, up(rows * 4) + 2 * up(rows * moves * 4)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_evict_keys_in_the_workspace_are_aligned(page):
    """Rows too long for shared memory keep their keys (and pool rows, one per four slots) in the
    workspace, one part per CTA. The parts are accessed 16 bytes at a time, so each takes a
    multiple of 16 bytes, whatever the capacity, and the workspace holds them all."""
    seen = set()
    for B, Hkv in ((1, 1), (1, 8), (3, 1), (2, 8), (4, 8), (8, 8), (5, 7), (16, 8), (80, 1)):
        for max_pages in [(41000 * n) // page + d for n in (1, 2, 4, 8, 10) for d in range(16)] + [8193, 5121]:
            c = cache(B=B, Hkv=Hkv, C=64, page=page, max_pages=max_pages, num_pages=8)
            rows, cluster, share, ahead = _evict_plan(B, Hkv, page, max_pages, 1000)
            got = xa._lib.xattn_cache_evict_workspace_size(c, 1000)
            if share <= 40960:                      # in shared memory
                assert got == ahead
                continue
            part = (4 * (share + share // 4) + 15) // 16 * 16
            assert got - ahead >= rows * cluster * part, (B, Hkv, max_pages)
            assert got - ahead < rows * cluster * part + 256
            if part != 5 * share:
                seen.add(cluster)
    # the shapes above do reach parts whose length alone is not a multiple of 16 bytes
    assert seen >= {16: {2, 4, 8}, 32: {4, 8}, 64: {8}, 128: set()}[page]

# ---------------------------------------------------- the binding's checks
def test_binding_checks_tensors():
    bf = dict(dtype=torch.bfloat16)
    pages, table, lens = torch.zeros(4, 2, 16, 64, **bf), torch.zeros(2, 2, dtype=torch.int32), \
        torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        xa.PagedCache(pages, pages, table, lens)
    with pytest.raises(TypeError):
        xa.PagedCache(pages.float(), pages.float(), table, lens)
    with pytest.raises(TypeError):
        xa.PagedCache(pages, pages, table.long(), lens)
    with pytest.raises(ValueError):
        xa.PagedCache(pages, pages[:, :1], table, lens)
    with pytest.raises(ValueError):
        xa.PagedCache(pages, pages, table, lens[:1])
    with pytest.raises(ValueError, match="scale"):
        xa.PagedCache(pages.to(torch.float8_e4m3fn), pages.to(torch.float8_e4m3fn), table, lens)
    with pytest.raises(ValueError, match="scale"):
        xa.PagedCache(pages, pages, table, lens, k_scale=torch.ones(2), v_scale=torch.ones(2))
    with pytest.raises(ValueError):
        xa.PagedCache(pages, pages, table, lens, acc=torch.zeros(4, 2, 8))
    with pytest.raises(TypeError):
        xa.PagedCache(pages, pages, table, lens, ordinal=torch.zeros(4, 2, 16))
    with pytest.raises(TypeError):
        xa.Rotary(torch.ones(32), (32,))
    with pytest.raises(ValueError):
        xa.Rotary(torch.ones(32, dtype=torch.float64), (16,))
    with pytest.raises(ValueError):
        xa.Rotary(torch.ones(0, dtype=torch.float64), ())
    with pytest.raises(ValueError, match="CUDA"):
        xa.Rotary(torch.ones(32, dtype=torch.float64), (32,))


def test_heads_of_strided_views():
    qkv = torch.zeros(2, 5, 12, 64, dtype=torch.bfloat16)
    h = xa._Heads.from_buffer_copy(xa._heads(qkv[:, :, 8:10].transpose(1, 2), "K"))
    assert (h.stride_b, h.stride_h, h.stride_m, h.heads) == (5 * 12 * 64, 64, 12 * 64, 2)
    assert h.data == qkv.data_ptr() + 8 * 64 * 2
    # a dimension of size 1 has no stride to speak of
    one = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16).as_strided((1, 1, 1, 64), (3, 5, 7, 1))
    assert xa._Heads.from_buffer_copy(xa._heads(one, "K")).stride_b == 0
    with pytest.raises(ValueError):
        xa._heads(qkv.transpose(2, 3), "K")
    with pytest.raises(TypeError):
        xa._heads(qkv.float(), "K")
    with pytest.raises(ValueError):
        xa._heads(qkv[0], "K")
