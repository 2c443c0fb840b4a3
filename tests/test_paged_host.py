"""Refusals of the paged cache's and the beam selection's calls (no GPU needed, no kernel launched)."""
import ctypes

import pytest
import torch

import speculative_decode_verify_gb300 as va
from speculative_decode_verify_gb300 import build as vbuild

FAKE, ODD = 0x1000, 0x1004     # never dereferenced: every call below is refused before any launch
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    vbuild.build()
    return va.lib()


def _pool(a):
    return [a["kc"], a["vc"], a["ks"], a["vs"]]


POOL = dict(kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, pages=100, heads=2)


def _append(L, **kw):
    a = dict(POOL, kn=FAKE, vn=FAKE, n=4, rows=6, live=FAKE, lens=FAKE, table=FAKE, width=10, fmt=0)
    a.update(kw)
    return L.kv_page_append_b8(a["kn"], a["vn"], a["n"], a["rows"], a["heads"], a["live"], a["lens"], a["table"], a["width"],
                               *_pool(a), a["pages"], a["fmt"], None, None)


def _attn(L, **kw):
    a = dict(POOL, q=FAKE, n=4, rows=6, group=6, live=FAKE, lens=FAKE, table=FAKE, width=10, fmt=1, window=0, scale=0.1,
             ws=FAKE, size=BIG, out=FAKE)
    a.update(kw)
    return L.verify_attn_paged_b8(a["q"], a["n"], a["rows"], a["heads"], a["group"], a["live"], a["lens"], a["table"],
                                  a["width"], *_pool(a), a["pages"], a["fmt"], a["window"], a["scale"], None, a["ws"],
                                  a["size"], a["out"], None, None, None)


def _extend(L, **kw):
    a = dict(POOL, table=FAKE, lens=FAKE, new=FAKE, n=4, width=10, refs=FAKE, layers=3, ws=FAKE, size=BIG)
    a.update(kw)
    return L.kv_page_extend(a["table"], a["lens"], a["new"], a["n"], a["width"], a["refs"], a["pages"], a["layers"],
                            a["heads"], *_pool(a), a["ws"], a["size"], None, None)


def _reorder(L, **kw):
    a = dict(table=FAKE, lens=FAKE, n=4, width=10, src=FAKE, group=2, refs=FAKE, pages=100)
    a.update(kw)
    return L.kv_page_reorder(a["table"], a["lens"], a["n"], a["width"], a["src"], a["group"], a["refs"], a["pages"], None,
                             None)


def _copy(L, **kw):
    a = dict(POOL, src=FAKE, dst=FAKE, n=4, layers=3)
    a.update(kw)
    return L.kv_page_copy(a["src"], a["dst"], a["n"], a["pages"], a["layers"], a["heads"], *_pool(a), None, None)


def _compact(L, **kw):
    a = dict(POOL, table=FAKE, n=4, width=10, refs=FAKE, layers=3, to=FAKE, live=FAKE, ws=FAKE, size=BIG)
    a.update(kw)
    return L.kv_page_compact(a["table"], a["n"], a["width"], a["refs"], a["pages"], a["layers"], a["heads"], *_pool(a),
                             a["to"], a["live"], a["ws"], a["size"], None, None)


def _beam(L, **kw):
    a = dict(x=FAKE, fmt=0, stride=160000, groups=2, beams=4, vocab=160000, scores=FAKE, fin=None, end=0, k=8, pa=FAKE,
             tk=FAKE, sc=FAKE, ws=FAKE, size=BIG)
    a.update(kw)
    return L.va_beam_select(a["x"], a["fmt"], a["stride"], a["groups"], a["beams"], a["vocab"], a["scores"], a["fin"],
                            a["end"], a["k"], a["pa"], a["tk"], a["sc"], a["ws"], a["size"], None)


POOL_BAD = [dict(kc=None), dict(vc=ODD), dict(ks=ODD), dict(vs=None), dict(pages=0), dict(heads=0), dict(heads=65)]
TABLE_BAD = [dict(table=None), dict(n=0), dict(n=1025), dict(width=0), dict(width=1 << 26)]


@pytest.mark.parametrize("kw", POOL_BAD + TABLE_BAD + [dict(kn=None), dict(vn=ODD), dict(rows=0), dict(rows=(1 << 24) + 1),
                                                       dict(live=None), dict(lens=None), dict(fmt=2), dict(fmt=-1)])
def test_append_refuses(L, kw):
    assert _append(L, **kw) == va.VA_INVALID_ARG


@pytest.mark.parametrize("kw", POOL_BAD + TABLE_BAD + [dict(q=None), dict(q=ODD), dict(rows=0), dict(rows=9), dict(group=0),
                                                       dict(group=9), dict(live=None), dict(lens=None), dict(fmt=2),
                                                       dict(window=-1), dict(scale=float("nan")), dict(ws=None),
                                                       dict(ws=ODD), dict(size=100), dict(out=None), dict(out=ODD)])
def test_attention_refuses(L, kw):
    assert _attn(L, **kw) == va.VA_INVALID_ARG


@pytest.mark.parametrize("kw", POOL_BAD + TABLE_BAD + [dict(lens=None), dict(new=None), dict(refs=None), dict(layers=0),
                                                       dict(ws=None), dict(ws=ODD), dict(size=255)])
def test_extend_refuses(L, kw):
    assert _extend(L, **kw) == va.VA_INVALID_ARG


@pytest.mark.parametrize("kw", TABLE_BAD + [dict(lens=None), dict(src=None), dict(refs=None), dict(group=-1), dict(group=3),
                                            dict(group=8), dict(pages=0)])
def test_reorder_refuses(L, kw):
    assert _reorder(L, **kw) == va.VA_INVALID_ARG


@pytest.mark.parametrize("kw", POOL_BAD + [dict(src=None), dict(dst=None), dict(n=-1), dict(n=101), dict(layers=0)])
def test_copy_refuses(L, kw):
    assert _copy(L, **kw) == va.VA_INVALID_ARG


@pytest.mark.parametrize("kw", POOL_BAD + TABLE_BAD + [dict(refs=None), dict(layers=0), dict(to=None), dict(live=None),
                                                       dict(ws=None), dict(ws=ODD), dict(size=255)])
def test_compact_refuses(L, kw):
    assert _compact(L, **kw) == va.VA_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(x=None), dict(x=ODD), dict(fmt=2), dict(stride=159996), dict(stride=160002),
                                dict(fmt=1, stride=160004), dict(groups=0), dict(groups=1025), dict(beams=0), dict(beams=33),
                                dict(vocab=0), dict(vocab=262145, stride=262148), dict(scores=None), dict(k=0), dict(k=33),
                                dict(fin=FAKE, end=-1), dict(fin=FAKE, end=160000), dict(pa=None), dict(tk=None),
                                dict(sc=None), dict(ws=None), dict(ws=ODD), dict(size=1000)])
def test_beam_refuses(L, kw):
    assert _beam(L, **kw) == va.VA_INVALID_ARG


def test_pools_past_32_bit_rows_are_unsupported(L):
    big = dict(pages=1 << 20, heads=64)                         # 2^32 rows of 128 bytes
    assert _append(L, **big) == _attn(L, **big) == _extend(L, **big) == _copy(L, **big) == _compact(L, **big) == va.VA_UNSUPPORTED
    assert _extend(L, n=1024, width=1 << 22) == va.VA_UNSUPPORTED
    assert _copy(L, n=0, src=None, dst=None) == va.VA_OK        # nothing to copy, nothing launched


def test_workspace_sizes(L):
    assert va.va_paged_workspace_bytes(0, 1, 1, 1) == va.va_paged_workspace_bytes(1025, 1, 1, 1) == 0
    assert va.va_paged_workspace_bytes(1, 9, 1, 1) == va.va_paged_workspace_bytes(1, 1, 65, 1) == 0
    assert va.va_paged_workspace_bytes(1, 1, 1, 9) == 0 and va.va_paged_workspace_bytes(4, 8, 2, 6) > 0
    # one workspace for the largest shape is large enough for smaller ones
    assert va.va_paged_workspace_bytes(1024, 8, 64, 8) >= va.va_paged_workspace_bytes(1, 1, 1, 1)
    assert va.va_page_ops_workspace_bytes(4, 10, 100) == 256 + 5 * 4 * 128
    assert va.va_page_ops_workspace_bytes(0, 10, 100) == va.va_page_ops_workspace_bytes(1025, 1, 1) == 0
    # per row the tiles' keys and statistics, then its scores and tokens, behind the counters
    assert va.va_beam_workspace_bytes(2, 4, 160000, 8) == 4 * (32768 + 1024) + 8 * (20 * (8 * 8 + 8) + 8 * 12)
    assert va.va_beam_workspace_bytes(1025, 1, 10, 1) == va.va_beam_workspace_bytes(1, 33, 10, 1) == 0
    assert va.va_beam_workspace_bytes(1, 1, 262145, 1) == va.va_beam_workspace_bytes(1, 1, 10, 33) == 0


def test_the_binding_refuses_shapes_that_do_not_fit():
    codes, scale = torch.zeros(5, 2, 64, 128, dtype=torch.uint8), torch.zeros(5, 2, 4)
    pool = [codes, codes.clone(), scale, scale.clone()]
    t, n = torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    new = torch.zeros(3, 2, 2, 128, dtype=torch.bfloat16)
    bad = [lambda: va.kv_page_append_b8(new[:, :, :1], new[:, :, :1], n, n, t, *pool),
           lambda: va.kv_page_append_b8(new, new, n[:2], n, t, *pool),
           lambda: va.kv_page_append_b8(new, new, n, n, t[:2], *pool),
           lambda: va.kv_page_append_b8(new.float(), new.float(), n, n, t, *pool),
           lambda: va.kv_page_append_b8(new.transpose(0, 1).contiguous().transpose(0, 1), new, n, n, t, *pool),
           lambda: va.kv_page_append_b8(new, new, n, n, t, codes, codes, scale[:, :1], scale),
           lambda: va.kv_page_append_b8(new, new, n, n, t, codes[..., :64], codes, scale, scale),
           lambda: va.kv_page_reorder(t, n, n[:1], n),
           lambda: va.kv_page_extend(t, n, n, n, *pool, codes),
           lambda: va.kv_page_copy(n, n[:2], *pool),
           lambda: va.verify_attn_paged_b8(new[..., :64].contiguous(), n, n, t, *pool, 0.1, None, codes, new),
           lambda: va.verify_attn_paged_b8(new, n, n, t, *pool, 0.1, torch.zeros(3), codes, new),
           lambda: va.va_beam_select(torch.zeros(4, 8), torch.zeros(3), 2, t[:2], t[:2], scale, codes),
           lambda: va.va_beam_select(torch.zeros(4, 8).double(), torch.zeros(4), 2, t[:2], t[:2], t[:2].float(), codes)]
    for call in bad:
        with pytest.raises(ValueError):
            call()


def _calls():
    """Every call with CPU tensors of the right shapes and types, by name: (function, arguments)."""
    f32, i32, b16 = torch.float32, torch.int32, torch.bfloat16
    codes, scale = torch.zeros(5, 2, 64, 128, dtype=torch.uint8), torch.zeros(5, 2, 4)
    pool = dict(k_codes=codes, v_codes=codes.clone(), k_scale=scale, v_scale=scale.clone())
    table, n, refs, one = (torch.zeros(s, dtype=i32) for s in ((3, 4), (3,), (5,), (1,)))
    new, q = torch.zeros(3, 2, 2, 128, dtype=b16), torch.zeros(3, 2, 4, 128, dtype=b16)
    ws, pick = torch.zeros(1 << 24, dtype=torch.uint8), torch.zeros(2, 3, dtype=i32)
    return {
        "append": (va.kv_page_append_b8, dict(k_new=new, v_new=new, n_live=n, lens=n, table=table, dev_status=one, **pool)),
        "attention": (va.verify_attn_paged_b8, dict(q=q, n_live=n, lens=n, table=table, scale=0.1, sink=torch.zeros(4),
                                                    workspace=ws, out=q, out_lse=torch.zeros(3, 2, 4), dev_status=one, **pool)),
        "extend": (va.kv_page_extend, dict(table=table, lens=n, n_new=n, refs=refs, workspace=ws, dev_status=one, **pool)),
        "reorder": (va.kv_page_reorder, dict(table=table, lens=n, src=n, refs=refs, dev_status=one)),
        "copy": (va.kv_page_copy, dict(src=n, dst=n, dev_status=one, **pool)),
        "compact": (va.kv_page_compact, dict(table=table, refs=refs, moved_to=refs, n_live_pages=one, workspace=ws,
                                             dev_status=one, **pool)),
        "beam": (va.va_beam_select, dict(logits=torch.zeros(8, 16), scores=torch.zeros(8), n_beams=4, parents=pick,
                                         tokens=pick, out_scores=torch.zeros(2, 3), workspace=ws,
                                         finished=torch.zeros(8, dtype=i32))),
    }


@pytest.mark.parametrize("name", sorted(_calls()))
def test_the_binding_refuses_tensors_that_are_on_no_gpu(name):
    call, args = _calls()[name]
    with pytest.raises(ValueError, match="have to be on a GPU"):
        call(**args)


@pytest.mark.parametrize("name", sorted(_calls()))
def test_the_binding_refuses_every_tensor_of_another_type(name):
    """Types of the same size among them: they would be read as what they are not."""
    call, args = _calls()[name]
    others = {torch.int32: [torch.float32, torch.uint32, torch.int64], torch.float32: [torch.int32, torch.float64, torch.bfloat16],
              torch.bfloat16: [torch.float16, torch.float32], torch.uint8: [torch.float8_e5m2, torch.bool, torch.float16]}
    tried = 0
    for key, t in args.items():
        if not torch.is_tensor(t) or key == "workspace":
            continue
        for kind in others[t.dtype]:
            if key == "logits" and kind is torch.bfloat16:
                continue
            wrong = dict(args, **{key: torch.zeros(t.shape).to(kind)})
            if key == "k_codes":
                wrong["v_codes"] = wrong[key]
            with pytest.raises(ValueError) as e:
                call(**wrong)
            assert "have to be on a GPU" not in str(e.value), (key, kind)
            tried += 1
    assert tried > 6


def test_the_binding_takes_bfloat16_bits_and_each_8_bit_code_type():
    """(as far as the check that comes last: these tensors are on no GPU)"""
    call, args = _calls()["append"]
    bits = args["k_new"].view(torch.int16)
    for kind in (torch.int8, torch.uint8, torch.float8_e4m3fn):
        codes = args["k_codes"].view(kind)
        with pytest.raises(ValueError, match="have to be on a GPU"):
            call(**dict(args, k_new=bits, v_new=bits, k_codes=codes, v_codes=codes))


def test_binding_constants_match_the_headers():
    import test_abi_host
    d = test_abi_host._defines()
    assert (d["VA_PAGED_MAX_SEQS"], d["VA_B8_BLOCK"]) == (va.PAGED_MAX_SEQS, va.B8_BLOCK)
    assert (d["VA_B8_E4M3"], d["VA_B8_INT8"]) == (va.B8_E4M3, va.B8_INT8)
    assert ctypes.sizeof(ctypes.c_void_p) == 8
