"""Refusals of the attention calls: argument errors come back before any HIP
call, and the binding checks what the C library cannot (no GPU needed)."""
import ctypes

import pytest
import torch

import speculative_decoding_verification_04_amd as sv

try:
    LIB = sv.library()
except RuntimeError:
    LIB = None

needs_lib = pytest.mark.skipif(LIB is None, reason="libspecverify.so not built")

# fake, never-dereferenced device addresses: validation fails before any use
P = [ctypes.c_void_p(0x10000000 * (i + 1)) for i in range(14)]
N = None
ODD = ctypes.c_void_p(0x10000008)


def _args(base, **kw):
    a = dict(base)
    for k in kw:
        assert k in a, k
    a.update(kw)
    return tuple(a.values())


MASK = dict(B=2, N=8, fc=P[0], ns=P[1], n=P[2], pos=P[3], mask=P[4], st=N, stream=N)
ROPE = dict(q=P[0], qs=256, k=P[1], ks=128, v=P[2], vs=128, kv=P[3], dt=1, L=1, B=2, H=2, C=64, D=64, layer=0, T=6,
            N=3, G=2, E=P[4], n=P[5], cu=N, pos=N, qw=N, kw=N, eps=1e-6, f=P[6], rot=64, near=0, out=P[7], st=N, s=N)
ROPE_P = dict(q=P[0], qs=256, k=P[1], ks=128, v=P[2], vs=128, kv=P[3], dt=1, L=1, pages=5, H=2, page=16, D=64, layer=0,
              T=6, B=2, N=3, G=2, table=P[4], most=4, n=P[5], cu=N, pos=N, qw=N, kw=N, eps=1e-6, f=P[6], rot=64, near=0,
              out=P[7], st=N, s=N)
PROMPT = dict(q=P[0], qs=256, kv=P[1], dt=1, L=2, B=2, H=2, C=64, D=64, layer=1, T=50, G=2, E=P[2], n=P[3], cu=P[4],
              scale=0.125, out=P[5], lse=N, st=N, s=N)
PROMPT_P = dict(q=P[0], qs=256, kv=P[1], dt=1, L=2, pages=9, H=2, page=16, D=64, layer=1, B=2, T=50, G=2, table=P[2],
                most=4, n=P[3], cu=P[4], scale=0.125, out=P[5], lse=N, st=N, s=N)
TREE = dict(q=P[0], qs=256, kv=P[1], dt=1, L=2, B=2, H=2, C=4096, D=64, layer=1, N=5, G=2, E=P[2], n=P[3], mask=N,
            scale=0.125, out=P[4], lse=N, st=N, ws=P[5], wsb=1 << 27, s=N)
TREE_P = dict(q=P[0], qs=256, kv=P[1], dt=1, L=2, pages=900, H=2, page=16, D=64, layer=1, B=2, N=5, G=2, table=P[2],
              most=256, n=P[3], mask=N, scale=0.125, out=P[4], lse=N, st=N, ws=P[5], wsb=1 << 27, s=N)


@needs_lib
@pytest.mark.parametrize("kw,code", [
    (dict(fc=N), sv.SPEC_EINVAL), (dict(ns=N), sv.SPEC_EINVAL), (dict(n=N), sv.SPEC_EINVAL),
    (dict(pos=N), sv.SPEC_EINVAL), (dict(mask=N), sv.SPEC_EINVAL), (dict(B=0), sv.SPEC_EINVAL),
    (dict(N=0), sv.SPEC_EINVAL), (dict(N=257), sv.SPEC_ECAPACITY), (dict(pos=P[0]), sv.SPEC_EINVAL),
    (dict(mask=P[3]), sv.SPEC_EINVAL), (dict(st=P[2]), sv.SPEC_EINVAL)])
def test_tree_mask_refusals(kw, code):
    assert LIB.spec_tree_mask(*_args(MASK, **kw)) == code


COMMON = [(dict(q=N), sv.SPEC_EINVAL), (dict(kv=N), sv.SPEC_EINVAL), (dict(n=N), sv.SPEC_EINVAL),
          (dict(out=N), sv.SPEC_EINVAL), (dict(dt=2), sv.SPEC_EINVAL), (dict(L=0), sv.SPEC_EINVAL),
          (dict(B=0), sv.SPEC_EINVAL), (dict(H=0), sv.SPEC_EINVAL), (dict(D=0), sv.SPEC_EINVAL),
          (dict(G=0), sv.SPEC_EINVAL), (dict(layer=-1), sv.SPEC_EINVAL), (dict(layer=2), sv.SPEC_EINVAL),
          (dict(D=60), sv.SPEC_EINVAL), (dict(D=264, qs=2112), sv.SPEC_ECAPACITY), (dict(qs=248), sv.SPEC_EINVAL),
          (dict(qs=257), sv.SPEC_EINVAL), (dict(q=ODD), sv.SPEC_EINVAL), (dict(kv=ODD), sv.SPEC_EINVAL),
          (dict(out=ODD), sv.SPEC_EINVAL), (dict(out=P[0]), sv.SPEC_EINVAL), (dict(out=P[1]), sv.SPEC_EINVAL),
          (dict(st=P[3]), sv.SPEC_EINVAL)]
SCALES = [(dict(scale=x), sv.SPEC_EINVAL) for x in (0.0, -1.0, float("nan"), float("inf"), 3e38)]
PAGES = [(dict(table=N), sv.SPEC_EINVAL), (dict(pages=0), sv.SPEC_EINVAL), (dict(page=0), sv.SPEC_EINVAL),
         (dict(most=0), sv.SPEC_EINVAL), (dict(most=1 << 28), sv.SPEC_EINVAL),
         (dict(most=1, page=2 ** 31 - 512), sv.SPEC_EINVAL)]
RECT = [(dict(E=N), sv.SPEC_EINVAL), (dict(C=0), sv.SPEC_EINVAL), (dict(C=2 ** 31 - 512), sv.SPEC_EINVAL)]


@needs_lib
@pytest.mark.parametrize("kw,code", COMMON + SCALES + RECT + [(dict(cu=N), sv.SPEC_EINVAL), (dict(T=0), sv.SPEC_EINVAL),
                                                              (dict(T=1 << 30), sv.SPEC_EINVAL)])
def test_prompt_refusals(kw, code):
    assert LIB.spec_prompt_attention(*_args(PROMPT, **kw)) == code


@needs_lib
@pytest.mark.parametrize("kw,code", COMMON + SCALES + PAGES + [(dict(cu=N), sv.SPEC_EINVAL), (dict(T=0), sv.SPEC_EINVAL)])
def test_prompt_paged_refusals(kw, code):
    assert LIB.spec_prompt_attention_paged(*_args(PROMPT_P, **kw)) == code


TREES = [(dict(N=0), sv.SPEC_EINVAL), (dict(N=257), sv.SPEC_ECAPACITY), (dict(ws=N), sv.SPEC_EWORKSPACE),
         (dict(wsb=1024), sv.SPEC_EWORKSPACE), (dict(ws=ctypes.c_void_p(0x60000010)), sv.SPEC_EWORKSPACE),
         (dict(ws=P[1]), sv.SPEC_EINVAL), (dict(mask=ctypes.c_void_p(0x70000002)), sv.SPEC_EINVAL),
         (dict(mask=P[4]), sv.SPEC_EINVAL)]


@needs_lib
@pytest.mark.parametrize("kw,code", COMMON + SCALES + RECT + TREES)
def test_tree_refusals(kw, code):
    assert LIB.spec_tree_attention(*_args(TREE, **kw)) == code


@needs_lib
@pytest.mark.parametrize("kw,code", COMMON + SCALES + PAGES + TREES)
def test_tree_paged_refusals(kw, code):
    assert LIB.spec_tree_attention_paged(*_args(TREE_P, **kw)) == code


ROPES = [(dict(q=N), sv.SPEC_EINVAL), (dict(k=N), sv.SPEC_EINVAL), (dict(v=N), sv.SPEC_EINVAL),
         (dict(kv=N), sv.SPEC_EINVAL), (dict(out=N), sv.SPEC_EINVAL), (dict(n=N), sv.SPEC_EINVAL),
         (dict(f=N), sv.SPEC_EINVAL), (dict(T=0), sv.SPEC_EINVAL), (dict(T=7), sv.SPEC_EINVAL),
         (dict(N=0), sv.SPEC_EINVAL), (dict(cu=P[8]), sv.SPEC_EINVAL), (dict(G=0), sv.SPEC_EINVAL),
         (dict(rot=63), sv.SPEC_EINVAL), (dict(rot=66), sv.SPEC_EINVAL), (dict(rot=-2), sv.SPEC_EINVAL),
         (dict(eps=-1.0), sv.SPEC_EINVAL), (dict(eps=float("nan")), sv.SPEC_EINVAL), (dict(D=60), sv.SPEC_EINVAL),
         (dict(D=264, qs=2112, ks=528, vs=528), sv.SPEC_ECAPACITY), (dict(ks=120), sv.SPEC_EINVAL),
         (dict(vs=129), sv.SPEC_EINVAL), (dict(k=ODD), sv.SPEC_EINVAL), (dict(out=P[3]), sv.SPEC_EINVAL),
         (dict(kv=P[1]), sv.SPEC_EINVAL), (dict(st=P[5]), sv.SPEC_EINVAL), (dict(layer=1), sv.SPEC_EINVAL),
         (dict(dt=9), sv.SPEC_EINVAL)]


@needs_lib
@pytest.mark.parametrize("kw,code", ROPES + RECT)
def test_rope_refusals(kw, code):
    assert LIB.spec_norm_rope_kv(*_args(ROPE, **kw)) == code


@needs_lib
@pytest.mark.parametrize("kw,code", ROPES + PAGES)
def test_rope_paged_refusals(kw, code):
    assert LIB.spec_norm_rope_kv_paged(*_args(ROPE_P, **kw)) == code


@needs_lib
def test_workspace_query():
    f = sv.spec_tree_attention_workspace_bytes
    assert f(2, 1, 8, 4, 128, 4096, sv.SPEC_BF16) > 0 and f(2, 1, 8, 4, 128, 4096, sv.SPEC_BF16) % 256 == 0
    assert f(2, 1, 8, 4, 128, 1, sv.SPEC_BF16) >= 16 * 32 * 128 * 4         # a slot for each piece
    for bad in [(0, 1, 8, 4, 128, 64), (1, 0, 8, 4, 128, 64), (1, 257, 8, 4, 128, 64), (1, 1, 0, 4, 128, 64),
                (1, 1, 8, 0, 128, 64), (1, 1, 8, 4, 257, 64), (1, 1, 8, 4, 128, 0)]:
        assert f(*bad, sv.SPEC_BF16) == 0
    assert f(2, 1, 8, 4, 128, 4096, 7) == 0


def test_binding_refuses_host_tensors_and_wrong_shapes():
    kv = torch.zeros(1, 2, 2, 2, 8, 64)
    q = torch.zeros(2, 3, 4, 64)
    with pytest.raises(ValueError, match="no whole group"):
        sv.spec_tree_attention(torch.zeros(2, 3, 3, 64), kv, 0, None, None, q, None)
    with pytest.raises(ValueError, match="must be on the GPU"):
        sv.spec_tree_attention(q, kv, 0, None, None, q, None)
    with pytest.raises(ValueError, match=r"\[B, N, heads, D\]"):
        sv.spec_tree_attention(q[0], kv, 0, None, None, q, None)
    with pytest.raises(ValueError, match=r"\[L, 2, planes, H, cols, D\]"):
        sv.spec_prompt_attention(q[0], kv[0], 0, None, None, None, q)
    with pytest.raises(ValueError, match="the cache must be contiguous"):
        sv.spec_norm_rope_kv(q, q[:, :, :2], q[:, :, :2], kv.transpose(4, 5).contiguous().transpose(4, 5), 0, None,
                             None, q)
    with pytest.raises(ValueError, match="must be on the GPU"):
        sv.spec_tree_mask(torch.zeros(1, 4, dtype=torch.int32), None, None, None, None)


def test_binding_checks_rows():
    """Layout checks of query rows (device -1: host tensors stand in)."""
    kv = torch.zeros(1, 2, 2, 2, 8, 64)
    wide = torch.zeros(2, 3, 8, 64)
    p, step, count = sv._token_rows(wide[:, :, :4], 4, kv, 64, "q", -1)
    assert (step, count) == (512, 6) and p == wide.data_ptr()
    assert sv._token_rows(wide[:, :1, :4], 4, kv, 64, "q", -1)[1:] == (1536, 2)     # one token a sequence
    assert sv._token_rows(wide[:1, :1, :4], 4, kv, 64, "q", -1)[1:] == (256, 1)
    for t, why in [(wide.bfloat16(), "must be torch.float32"), (wide[:, :, :3], r"must be \[\.\.\., 4, 64\]"),
                   (wide[:, :, ::2], "contiguous"), (wide[:, :2, :4], "one stride"),
                   (wide.transpose(2, 3)[:, :, :4, :].expand(2, 3, 4, 8), "must be")]:
        with pytest.raises(ValueError, match=why):
            sv._token_rows(t, 4, kv, 64, "q", -1)
    with pytest.raises(ValueError, match="needs 5 tokens, has 6"):
        sv._token_rows(wide[:, :, :4], 4, kv, 64, "k", -1, 5)
    t = torch.zeros(8, dtype=torch.int32)
    assert sv._need(None, torch.int32, 1, "mask", -1, True) is None
    for args, why in [((None, torch.int32, 1, "kv_len", -1), "kv_len is required"),
                      ((t, torch.int64, 1, "kv_len", -1), "must be torch.int64"),
                      ((t, torch.int32, 9, "kv_len", -1), "at least 9 elements"),
                      ((t, torch.int32, 8, "kv_len", 0), "must be on cuda:0"),
                      ((t[::2], torch.int32, 4, "kv_len", -1), "must be contiguous")]:
        with pytest.raises(ValueError, match=why):
            sv._need(*args)


# addresses 16 TB apart, so that sizes near the limits do not overlap
FAR = [ctypes.c_void_p((i + 1) << 44) for i in range(9)]


@needs_lib
@pytest.mark.parametrize("B,N", [(1 << 24, 256), (1 << 25, 65), (1 << 26, 1), (2 ** 31 - 1, 64)])
def test_tree_mask_refuses_launches_past_32_bits(B, N):
    assert LIB.spec_tree_mask(B, N, *FAR[:5], None, None) == sv.SPEC_EINVAL


@needs_lib
@pytest.mark.parametrize("T,G,st", [(1 << 24, 254, N), (1 << 26, 1, N), ((1 << 24) - 1, 254, FAR[8])])
def test_rope_refuses_launches_past_32_bits(T, G, st):
    """A workgroup of 64 lanes (3 heads of one lane each) or 256 (256 heads) a token, and some for the status."""
    big = dict(q=FAR[0], qs=8 * G, k=FAR[1], ks=8, v=FAR[2], vs=8, kv=FAR[3], H=1, D=8, rot=8, G=G, T=T, out=FAR[5])
    assert LIB.spec_norm_rope_kv(*_args(ROPE, **big, B=1, N=T, C=64, E=FAR[6], n=FAR[7], f=FAR[4], st=st)) == sv.SPEC_EINVAL
    assert LIB.spec_norm_rope_kv_paged(*_args(ROPE_P, **big, B=1, N=T, table=FAR[6], n=FAR[7], f=FAR[4], st=st)) == sv.SPEC_EINVAL


@needs_lib
@pytest.mark.parametrize("B,T,H", [(1 << 24, 5, 1), (1 << 20, 5, 16), (1, (2 ** 31 - 2) // 2, 2)])
def test_prompts_refuse_launches_past_32_bits(B, T, H):
    big = dict(q=FAR[0], qs=16 * H, kv=FAR[1], L=1, layer=0, H=H, D=8, T=T, n=FAR[3], cu=FAR[4], out=FAR[5], B=B)
    assert LIB.spec_prompt_attention(*_args(PROMPT, **big, C=8, E=FAR[2])) == sv.SPEC_EINVAL
    assert LIB.spec_prompt_attention_paged(*_args(PROMPT_P, **big, table=FAR[2], most=1)) == sv.SPEC_EINVAL


@needs_lib
@pytest.mark.parametrize("B,nodes,H,G", [(1 << 10, 256, 1, 256), (1 << 25, 1, 1, 2), (1 << 24, 1, 1, 1), (1 << 20, 2, 16, 1)])
def test_trees_refuse_launches_past_32_bits(B, nodes, H, G):
    """2^26 query rows need 2^32 lanes to join; 2^24 pieces as many to attend.  The workspace query says 0."""
    assert sv.spec_tree_attention_workspace_bytes(B, nodes, H, G, 8, 512, sv.SPEC_BF16) == 0
    big = dict(q=FAR[0], qs=8 * H * G, kv=FAR[1], L=1, layer=0, H=H, D=8, N=nodes, G=G, n=FAR[3], out=FAR[4], B=B,
               ws=FAR[5], wsb=1 << 43)
    assert LIB.spec_tree_attention(*_args(TREE, **big, C=512, E=FAR[2])) == sv.SPEC_EINVAL
    assert LIB.spec_tree_attention_paged(*_args(TREE_P, **big, table=FAR[2], most=32)) == sv.SPEC_EINVAL


@needs_lib
def test_the_largest_tree_calls_that_fit():
    """Just below: the query names a size, and the checks end at the workspace (its size is not enough)."""
    assert sv.spec_tree_attention_workspace_bytes((1 << 10) - 1, 256, 1, 256, 8, 512, sv.SPEC_BF16) > 0
    big = dict(q=FAR[0], qs=8 * 256, kv=FAR[1], L=1, layer=0, H=1, D=8, N=256, G=256, n=FAR[3], out=FAR[4],
               B=(1 << 10) - 1, ws=FAR[5], wsb=256)
    assert LIB.spec_tree_attention(*_args(TREE, **big, C=512, E=FAR[2])) == sv.SPEC_EWORKSPACE


@needs_lib
def test_tile_counts_stay_below_31_bits_with_the_target_added():
    big = dict(q=FAR[0], qs=8, kv=FAR[1], L=1, layer=0, H=1, D=8, N=1, G=1, n=FAR[3], out=FAR[4], ws=FAR[5], wsb=1 << 43)
    tiles = (2 ** 31 - 100) // 129                        # of 128 rows: 129 sequences have 2^31 - 137, a target is 256
    for each, code in [(tiles, sv.SPEC_EINVAL), (tiles - 2, sv.SPEC_EWORKSPACE)]:
        args = dict(big, wsb=256, B=129, table=FAR[2], most=each * 8, pages=9, page=16)
        assert LIB.spec_tree_attention_paged(*_args(TREE_P, **args)) == code
