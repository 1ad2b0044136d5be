"""Refusals of the calls on caches of 4-bit numbers and of the tree commit over
pages: argument errors come back before any HIP call (no GPU needed)."""
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
P = [ctypes.c_void_p(0x10000000 * (i + 1)) for i in range(15)]
N = None
EINVAL, ECAPACITY, EWORKSPACE = sv.SPEC_EINVAL, sv.SPEC_ECAPACITY, sv.SPEC_EWORKSPACE


def odd(i, by=8):
    return ctypes.c_void_p(0x10000000 * (i + 1) + by)


ROPE = dict(q=P[0], qs=256, k=P[1], ks=128, v=P[2], vs=128, c=P[3], sc=P[9], dt=1, L=1, B=2, H=2, C=64, D=64, layer=0,
            T=6, N=3, G=2, E=P[4], n=P[5], cu=N, pos=N, qw=N, kw=N, eps=1e-6, f=P[6], rot=64, near=0, out=P[7], st=N,
            s=N)
ROPE_P = dict(q=P[0], qs=256, k=P[1], ks=128, v=P[2], vs=128, c=P[3], sc=P[9], dt=1, L=1, pages=5, H=2, page=16, D=64,
              layer=0, T=6, B=2, N=3, G=2, table=P[4], most=4, n=P[5], cu=N, pos=N, qw=N, kw=N, eps=1e-6, f=P[6],
              rot=64, near=0, out=P[7], st=N, s=N)
UNPACK = dict(c=P[3], sc=P[9], dt=1, L=2, B=2, H=2, C=64, D=64, layer=1, T=6, N=3, E=P[4], n=P[5], cu=N, ko=P[7],
              vo=P[8], st=N, s=N)
UNPACK_P = dict(c=P[3], sc=P[9], dt=1, L=2, pages=5, H=2, page=16, D=64, layer=1, T=6, B=2, N=3, table=P[4], most=4,
                n=P[5], cu=N, ko=P[7], vo=P[8], st=N, s=N)
PROMPT = dict(q=P[0], qs=256, c=P[3], sc=P[9], dt=1, L=2, B=2, H=2, C=64, D=64, layer=1, T=50, G=2, E=P[4], n=P[5],
              cu=P[6], scale=0.125, out=P[7], lse=N, st=N, s=N)
PROMPT_P = dict(q=P[0], qs=256, c=P[3], sc=P[9], dt=1, L=2, pages=9, H=2, page=16, D=64, layer=1, B=2, T=50, G=2,
                table=P[4], most=4, n=P[5], cu=P[6], scale=0.125, out=P[7], lse=N, st=N, s=N)
TREE = dict(q=P[0], qs=256, c=P[3], sc=P[9], dt=1, L=2, B=2, H=2, C=4096, D=64, layer=1, N=5, G=2, E=P[4], n=P[5],
            mask=N, scale=0.125, out=P[7], lse=N, st=N, ws=P[10], wsb=1 << 27, s=N)
TREE_P = dict(q=P[0], qs=256, c=P[3], sc=P[9], dt=1, L=2, pages=900, H=2, page=16, D=64, layer=1, B=2, N=5, G=2,
              table=P[4], most=256, n=P[5], mask=N, scale=0.125, out=P[7], lse=N, st=N, ws=P[10], wsb=1 << 27, s=N)
COMPACT = dict(pool=P[3], dt=1, L=2, pages=9, H=2, page=16, D=64, B=2, N=5, table=P[4], most=4, n=P[5], path=P[6],
               e=P[7], st=N, s=N)

# of every call on such a cache
COMMON = [(dict(c=N), EINVAL), (dict(sc=N), EINVAL), (dict(n=N), EINVAL), (dict(dt=2), EINVAL), (dict(dt=-1), EINVAL),
          (dict(L=0), EINVAL), (dict(B=0), EINVAL), (dict(H=0), EINVAL), (dict(D=0), EINVAL), (dict(layer=-1), EINVAL),
          (dict(layer=2), EINVAL), (dict(D=32), EINVAL), (dict(D=96), EINVAL), (dict(D=80), EINVAL),
          (dict(c=odd(3)), EINVAL), (dict(sc=odd(9, 4)), EINVAL), (dict(T=0), EINVAL)]
BOTH = [(dict(sc=P[3]), EINVAL), (dict(sc=ctypes.c_void_p(0x40000000 + 64)), EINVAL)]   # codes and scales overlap
RECT = [(dict(E=N), EINVAL), (dict(C=0), EINVAL), (dict(C=2 ** 31 - 512), EINVAL)]
PAGES = [(dict(table=N), EINVAL), (dict(pages=0), EINVAL), (dict(page=0), EINVAL), (dict(most=0), EINVAL),
         (dict(most=1 << 28), EINVAL)]
QUERIES = [(dict(q=N), EINVAL), (dict(out=N), EINVAL), (dict(G=0), EINVAL), (dict(qs=248), EINVAL),
           (dict(qs=257), EINVAL), (dict(q=odd(0)), EINVAL), (dict(out=odd(7)), EINVAL), (dict(out=P[0]), EINVAL),
           (dict(out=P[3]), EINVAL), (dict(out=P[9]), EINVAL), (dict(st=P[5]), EINVAL), (dict(st=P[9]), EINVAL),
           (dict(D=320, qs=2560, ks=1280, vs=1280), ECAPACITY)]
SCALES = [(dict(scale=x), EINVAL) for x in (0.0, -1.0, float("nan"), float("inf"), 3e38)]
ROPES = [(dict(k=N), EINVAL), (dict(v=N), EINVAL), (dict(f=N), EINVAL), (dict(T=7), EINVAL), (dict(N=0), EINVAL),
         (dict(cu=P[8]), EINVAL), (dict(rot=63), EINVAL), (dict(rot=66), EINVAL), (dict(eps=-1.0), EINVAL),
         (dict(ks=120), EINVAL), (dict(vs=129), EINVAL), (dict(k=odd(1)), EINVAL), (dict(c=P[1]), EINVAL),
         (dict(sc=P[2]), EINVAL), (dict(layer=1), EINVAL)] + BOTH
UNPACKS = [(dict(ko=N), EINVAL), (dict(vo=N), EINVAL), (dict(T=7), EINVAL), (dict(N=0), EINVAL), (dict(cu=P[0]), EINVAL),
           (dict(ko=odd(7)), EINVAL), (dict(vo=odd(8, 4)), EINVAL), (dict(ko=P[3]), EINVAL), (dict(vo=P[9]), EINVAL),
           (dict(vo=P[7]), EINVAL), (dict(st=P[5]), EINVAL), (dict(st=P[7]), EINVAL), (dict(D=320), ECAPACITY),
           (dict(H=1 << 20), EINVAL)]
TREES = [(dict(N=0), EINVAL), (dict(N=257), ECAPACITY), (dict(ws=N), EWORKSPACE), (dict(wsb=1024), EWORKSPACE),
         (dict(ws=ctypes.c_void_p(0xB0000010)), EWORKSPACE), (dict(ws=P[3]), EINVAL), (dict(ws=P[9]), EINVAL),
         (dict(mask=odd(11, 2)), EINVAL), (dict(mask=P[7]), EINVAL)]
PROMPTS = [(dict(cu=N), EINVAL), (dict(T=1 << 30), EINVAL)]
CALLS = {
    "spec_norm_rope_kv_mx": (ROPE, COMMON + QUERIES + ROPES + RECT),
    "spec_norm_rope_kv_mx_paged": (ROPE_P, COMMON + QUERIES + ROPES + PAGES),
    "spec_unpack_kv_mx": (UNPACK, COMMON + UNPACKS + RECT),
    "spec_unpack_kv_mx_paged": (UNPACK_P, COMMON + UNPACKS + PAGES),
    "spec_prompt_attention_mx": (PROMPT, COMMON + QUERIES + SCALES + PROMPTS + RECT),
    "spec_prompt_attention_mx_paged": (PROMPT_P, COMMON + QUERIES + SCALES + PROMPTS + PAGES),
    "spec_tree_attention_mx": (TREE, COMMON + QUERIES + SCALES + TREES + RECT),
    "spec_tree_attention_mx_paged": (TREE_P, COMMON + QUERIES + SCALES + TREES + PAGES),
    "spec_compact_tree_paged": (COMPACT, [
        (dict(pool=N), EINVAL), (dict(table=N), EINVAL), (dict(n=N), EINVAL), (dict(path=N), EINVAL),
        (dict(e=N), EINVAL), (dict(dt=2), EINVAL), (dict(L=0), EINVAL), (dict(pages=0), EINVAL), (dict(H=0), EINVAL),
        (dict(page=0), EINVAL), (dict(D=0), EINVAL), (dict(B=0), EINVAL), (dict(N=0), EINVAL),
        (dict(N=257), ECAPACITY), (dict(most=0), EINVAL), (dict(most=1 << 28), EINVAL), (dict(pool=odd(3, 1)), EINVAL),
        (dict(st=odd(11, 2)), EINVAL), (dict(st=P[3]), EINVAL), (dict(st=P[7]), EINVAL), (dict(path=P[3]), EINVAL),
        (dict(D=1 << 23), EINVAL), (dict(H=1 << 30), EINVAL), (dict(L=1 << 30), EINVAL), (dict(L=1 << 24), EINVAL)]),
}


@needs_lib
@pytest.mark.parametrize("name,kw,code", [
    pytest.param(name, kw, code, id=f"{name}-{'-'.join(f'{k}={v}' for k, v in kw.items())}")
    for name, (base, cases) in CALLS.items() for kw, code in cases if all(k in base for k in kw) or "qs" in kw])
def test_refusals(name, kw, code):
    base = dict(CALLS[name][0])
    for k, v in kw.items():
        if k in base:
            base[k] = v
        else:
            assert k in ("ks", "vs", "qs"), k
    assert getattr(LIB, name)(*base.values()) == code


@needs_lib
def test_workspace_query():
    f = sv.spec_tree_attention_mx_workspace_bytes
    assert f(2, 5, 4, 7, 128, 4096, sv.SPEC_BF16) % 256 == 0
    assert f(2, 5, 4, 7, 128, 4096, sv.SPEC_BF16) > 0 and f(2, 5, 4, 7, 128, 4096, sv.SPEC_F32) > 0
    for bad in [(0, 5, 4, 7, 128, 4096, 1), (2, 0, 4, 7, 128, 4096, 1), (2, 257, 4, 7, 128, 4096, 1),
                (2, 5, 0, 7, 128, 4096, 1), (2, 5, 4, 0, 128, 4096, 1), (2, 5, 4, 7, 96, 4096, 1),
                (2, 5, 4, 7, 320, 4096, 1), (2, 5, 4, 7, 0, 4096, 1), (2, 5, 4, 7, 128, 0, 1), (2, 5, 4, 7, 128, 4096, 2),
                (1 << 20, 256, 8, 8, 128, 4096, 1)]:
        assert f(*bad) == 0, bad


def test_binding_checks_codes_and_scales():
    codes, scales = torch.zeros(1, 2, 3, 2, 16, 64, dtype=torch.uint8), torch.zeros(1, 2, 3, 2, 16, 4, dtype=torch.uint8)
    assert sv._mx_dims(codes, scales, 8) == (1, 3, 2, 16, 128, 4)
    for c, s in ((codes, scales[..., :2]), (codes[..., :48].contiguous(), scales[..., :3].contiguous()),
                 (codes, scales[:, :1]), (codes[0], scales[0])):
        with pytest.raises(ValueError):
            sv._mx_dims(c, s, 8)
    with pytest.raises(ValueError):
        sv._mx_dims(codes, scales, 3)                      # no whole group
    q = torch.zeros(3, 1, 8, 128, dtype=torch.bfloat16)
    i32 = torch.zeros(3, 4, dtype=torch.int32)
    for call in (lambda: sv.spec_tree_attention_mx(q, codes, scales, 0, i32[:1, 0], i32[:, 0], q, None),
                 lambda: sv.spec_prompt_attention_mx_paged(q[:, 0], codes, scales, 0, i32[0], i32, i32[:, 0], q),
                 lambda: sv.spec_norm_rope_kv_mx(q, q, q, codes, scales, 0, i32[:1, 0], i32[:, 0], q),
                 lambda: sv.spec_unpack_kv_mx(codes, scales, 0, i32[:1, 0], i32[:, 0], q, q),
                 lambda: sv.spec_compact_tree_paged(q.view(1, 1, 1, 3, 8, 128).expand(1, 2, 1, 3, 8, 128), i32, i32[:, 0],
                                                    i32, i32[:, 0])):
        with pytest.raises(ValueError, match="on the GPU"):
            call()
    with pytest.raises(ValueError, match="pool must be"):
        sv.spec_compact_tree_paged(codes[0], i32, i32[:, 0], i32, i32[:, 0])
