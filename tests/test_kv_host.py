"""Refusals of the rotary, cache and expert-layer calls (CPU only: every call here is refused before it
reaches a device)."""
from __future__ import annotations

import ctypes

import pytest
import torch

from bit_quantized_matmul_amd import binding as B

P = ctypes.c_void_p(4096)                             # never dereferenced: the checks fail first
ODD = ctypes.c_void_p(4097)
OFF8 = ctypes.c_void_p(4104)                          # 8-byte aligned only
EINVAL, EALIGN, ENOTSUP = B.BQM_EINVAL, B.BQM_EALIGN, B.BQM_ENOTSUP


@pytest.fixture(scope="module")
def lib():
    return B.load_library()


ROPE = dict(x=P, dtype=1, tokens=4, heads=2, dim=64, xt=128, xh=64, positions=P, freqs=P, rotary=64, interleaved=0,
            mscale=1.0, backward=0, y=P, yt=128, yh=64, stream=None)
APPEND = dict(k=P, v=P, dtype=1, tokens=4, heads=2, dim=64, kt=128, kh=64, vt=128, vh=64, offsets=None, lens=P, seqs=4,
              pages=P, stride=3, width=3, positions=P, freqs=P, rotary=64, interleaved=0, mscale=1.0, kc=P, vc=P, ks=P,
              vs=P, count=9, stream=None)
ATTEND = dict(q=P, dtype=1, tokens=4, heads=8, dim=64, qt=512, qh=64, offsets=None, lens=P, seqs=4, pages=P, stride=3,
              width=3, kc=P, vc=P, ks=P, vs=P, count=9, kv_heads=2, scale=0.1, window=0, out=P, ws=P, nws=1 << 40,
              stream=None)
MOE = dict(x=P, dtype=1, tokens=4, hidden=256, xs=256, logits=P, ldtype=0, ls=8, experts=8, top=2, renorm=1, w13=P, s13=P,
           w2=P, s2=P, ffn=128, out=P, ws=P, nws=1 << 40, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(x=None), EINVAL), (dict(y=None), EINVAL), (dict(positions=None), EINVAL), (dict(freqs=None), EINVAL),
    (dict(dtype=3), EINVAL), (dict(tokens=0), EINVAL), (dict(heads=0), EINVAL), (dict(dim=0), EINVAL),
    (dict(rotary=0), EINVAL), (dict(rotary=63), EINVAL), (dict(rotary=66), EINVAL), (dict(rotary=-2), EINVAL),
    (dict(xt=127), EINVAL), (dict(xh=63), EINVAL), (dict(yt=0), EINVAL), (dict(yt=64, yh=64), EINVAL),
    (dict(xt=256), EINVAL),                                            # in place, other strides
    (dict(dim=1025, rotary=64, xt=1 << 20, xh=2048, yt=1 << 20, yh=2048), ENOTSUP),
    (dict(tokens=1 << 24), ENOTSUP), (dict(heads=65536, xt=1 << 23, yt=1 << 23), ENOTSUP),
    (dict(x=ODD), EALIGN), (dict(y=ODD), EALIGN), (dict(positions=ODD), EALIGN), (dict(freqs=ctypes.c_void_p(4100)), EALIGN),
])
def test_rope_refuses(lib, change, code):
    assert lib.rope(*{**ROPE, **change}.values()) == code


@pytest.mark.parametrize("change,code", [
    *[({name: None}, EINVAL) for name in ("k", "v", "lens", "pages", "kc", "vc", "ks", "vs", "positions", "freqs")],
    (dict(dtype=7), EINVAL), (dict(tokens=0), EINVAL), (dict(heads=0), EINVAL), (dict(dim=0), EINVAL), (dict(seqs=0), EINVAL),
    (dict(width=0), EINVAL), (dict(count=0), EINVAL), (dict(stride=2), EINVAL), (dict(rotary=65), EINVAL),
    (dict(rotary=66), EINVAL), (dict(tokens=5), EINVAL), (dict(kt=64), EINVAL), (dict(vh=32), EINVAL),
    (dict(dim=257, rotary=0, kt=1 << 20, kh=512, vt=1 << 20, vh=512), ENOTSUP), (dict(width=1 << 25, stride=1 << 25), ENOTSUP),
    (dict(heads=65536, kt=1 << 23, vt=1 << 23), ENOTSUP),
    (dict(tokens=1 << 24, seqs=1 << 24), ENOTSUP), (dict(tokens=1 << 30, seqs=4, offsets=P), ENOTSUP),
    (dict(kc=OFF8), EALIGN), (dict(vc=OFF8), EALIGN), (dict(k=ODD), EALIGN), (dict(v=ODD), EALIGN), (dict(ks=ODD), EALIGN),
    (dict(vs=ODD), EALIGN), (dict(lens=ODD), EALIGN), (dict(pages=ODD), EALIGN), (dict(offsets=ODD), EALIGN),
    (dict(positions=ODD), EALIGN), (dict(freqs=ctypes.c_void_p(4100)), EALIGN),
])
def test_append_refuses(lib, change, code):
    assert lib.kv_append(*{**APPEND, **change}.values()) == code


@pytest.mark.parametrize("change,code", [
    *[({name: None}, EINVAL) for name in ("q", "lens", "pages", "kc", "vc", "ks", "vs", "out")],
    (dict(dtype=-1), EINVAL), (dict(tokens=0), EINVAL), (dict(heads=0), EINVAL), (dict(heads=7), EINVAL), (dict(kv_heads=0), EINVAL),
    (dict(dim=0), EINVAL), (dict(seqs=0), EINVAL), (dict(width=0), EINVAL), (dict(count=0), EINVAL), (dict(stride=2), EINVAL),
    (dict(window=-1), EINVAL), (dict(tokens=5), EINVAL), (dict(qt=511), EINVAL), (dict(qh=63), EINVAL),
    (dict(dim=257, qt=1 << 20, qh=512), ENOTSUP), (dict(width=1 << 25, stride=1 << 25), ENOTSUP),
    (dict(tokens=1 << 21, seqs=1 << 21), ENOTSUP),
    (dict(kc=OFF8), EALIGN), (dict(vc=OFF8), EALIGN), (dict(q=ODD), EALIGN), (dict(out=ODD), EALIGN), (dict(ks=ODD), EALIGN),
    (dict(vs=ODD), EALIGN), (dict(lens=ODD), EALIGN), (dict(offsets=ODD), EALIGN), (dict(ws=OFF8), EALIGN),
])
def test_attention_refuses(lib, change, code):
    assert lib.kv_attention(*{**ATTEND, **change}.values()) == code


@pytest.mark.parametrize("change,code", [
    *[({name: None}, EINVAL) for name in ("x", "logits", "w13", "s13", "w2", "s2", "out")],
    (dict(dtype=3), EINVAL), (dict(ldtype=3), EINVAL), (dict(tokens=0), EINVAL), (dict(hidden=0), EINVAL), (dict(ffn=0), EINVAL),
    (dict(experts=0), EINVAL), (dict(top=0), EINVAL), (dict(top=9), EINVAL), (dict(xs=255), EINVAL), (dict(ls=7), EINVAL),
    (dict(nws=0), EINVAL), (dict(ws=None), EINVAL),
    (dict(tokens=33), ENOTSUP), (dict(experts=1025, ls=1025), ENOTSUP), (dict(experts=64, ls=64, top=33), ENOTSUP),
    (dict(hidden=65537, xs=65537), ENOTSUP), (dict(ffn=65537), ENOTSUP),
    (dict(w13=OFF8), EALIGN), (dict(w2=OFF8), EALIGN), (dict(ws=OFF8), EALIGN), (dict(x=ODD), EALIGN), (dict(out=ODD), EALIGN),
    (dict(logits=ODD), EALIGN), (dict(s13=ODD), EALIGN), (dict(s2=ODD), EALIGN),
])
def test_expert_layer_refuses(lib, change, code):
    assert lib.moe_ffn(*{**MOE, **change}.values()) == code


def test_workspaces(lib):
    n = ctypes.c_int64()
    assert lib.kv_attention_workspace(4, 4, 8, 2, 64, 3, None) == EINVAL
    assert lib.kv_attention_workspace(4, 4, 8, 3, 64, 3, ctypes.byref(n)) == EINVAL
    assert lib.kv_attention_workspace(4, 4, 8, 2, 64, 3, ctypes.byref(n)) == B.BQM_OK and n.value >= 0
    assert lib.moe_ffn_workspace(4, 8, 2, 256, 128, None) == EINVAL
    assert B.moe_ffn_workspace(4, 8, 2, 256, 128) > 0
    with pytest.raises(B.BqmError):
        B.moe_ffn_workspace(33, 8, 2, 256, 128)


def test_binding_refuses_shapes_types_and_devices():
    f8, i32 = torch.float8_e4m3fn, torch.int32
    x, f, p = torch.zeros(4, 2, 64), torch.zeros(32, dtype=torch.float64), torch.zeros(4, dtype=i32)
    for args, match in (((x[0], p, f), "tokens, heads, dim"), ((x.double(), p, f), "float32, bfloat16 or float16"),
                        ((x, p[:3], f), "positions"), ((x, p, torch.zeros(33, dtype=torch.float64)), "freqs"),
                        ((x, p, None), "freqs"), ((x.transpose(1, 2), p, f), "contiguous|freqs"), ((x, p, f), "CUDA"),
                        ((x[:0], p[:0], f), "tokens, heads, dim")):
        with pytest.raises(ValueError, match=match):
            B.rope(*args)
    cache = B.kv_cache(3, 2, 50, device="cpu")
    assert cache.k.shape == (3, 2, 64, 64) and cache.v.shape == (3, 2, 64, 64) and cache.k.dtype == f8
    k, pages, lens = torch.zeros(4, 2, 50), torch.zeros(4, 2, dtype=i32), torch.zeros(4, dtype=i32)
    with pytest.raises(ValueError, match="CUDA"):
        B.kv_append(cache, k, k, pages, lens)
    with pytest.raises(ValueError, match="v must have shape"):
        B.kv_append(cache, k, k[:3], pages, lens)
    with pytest.raises(ValueError, match="cache.k must have shape"):
        B.kv_append(cache, torch.zeros(4, 2, 70), torch.zeros(4, 2, 70), pages, lens)
    with pytest.raises(ValueError, match="cache's 2 heads"):
        B.kv_append(cache, torch.zeros(4, 3, 50), torch.zeros(4, 3, 50), pages, lens)
    with pytest.raises(ValueError, match="without offsets"):
        B.kv_append(cache, k[:3], k[:3], pages, lens)
    with pytest.raises(ValueError, match="offsets must have shape"):
        B.kv_append(cache, k, k, pages, lens, offsets=lens)
    with pytest.raises(ValueError, match="positions come with freqs"):
        B.kv_append(cache, k, k, pages, lens, positions=lens)
    with pytest.raises(ValueError, match="v_scale"):
        B.kv_append(cache._replace(v_scale=cache.v_scale[:2]), k, k, pages, lens)
    with pytest.raises(ValueError, match="multiple of the cache's 2"):
        B.kv_attention(torch.zeros(4, 3, 50), cache, pages, lens)
    with pytest.raises(ValueError, match="window"):
        B.kv_attention(torch.zeros(4, 4, 50), cache, pages, lens, window=-1)
    with pytest.raises(ValueError, match="CUDA"):
        B.kv_attention(torch.zeros(4, 4, 50), cache, pages, lens)
    with pytest.raises(ValueError, match="pages must have shape"):
        B.kv_attention(torch.zeros(4, 4, 50), cache, pages[0], lens)
    for dim in (0, 257):
        with pytest.raises(ValueError, match="1 .. 256"):
            B.kv_cache(1, 1, dim, device="cpu")
    x, logits = torch.zeros(4, 100), torch.zeros(4, 3)
    w13, s13 = torch.zeros(3, 40, 128, dtype=f8), torch.zeros(3, 1, 1)
    w2, s2 = torch.zeros(3, 100, 128, dtype=f8), torch.zeros(3, 1, 1)
    for change, match in ((dict(logits=logits[:3]), "logits must have shape"), (dict(w13=w13[:2]), "w13 must have shape"),
                          (dict(w13=w13[:, :39]), "w13 must have shape"), (dict(w2=w2[:, :99]), "w2 must have shape"),
                          (dict(w13_scale=s13[:2]), "w13_scale"), (dict(w2_scale=s2[:2]), "w2_scale"), (dict(), "CUDA")):
        with pytest.raises(ValueError, match=match):
            B.moe_ffn(**{**dict(x=x, w13=w13, w13_scale=s13, w2=w2, w2_scale=s2, logits=logits, top=2), **change})
