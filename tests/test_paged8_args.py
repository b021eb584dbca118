"""Refusals of the operators on 8-bit pages and of token log probabilities (no GPU: what the host checks is refused
before any device work, so fake aligned addresses stand in for device memory)."""
import pathlib
import re

import pytest
import torch

from tests.test_paged_args import ATTN, NORM, P, L, refused  # noqa: F401

NORM8 = dict(NORM, kscale=P, vscale=P)
ATTN8 = dict(ATTN, kscale=P, vscale=P)
SCORE = dict(stream=0, N=4, V=1000, logits=P, logits_dtype=2, ld=1000, tokens=P, top=5, logprobs=P, entropy=P, top_ids=P,
             top_logprobs=P)


@pytest.mark.parametrize("change", [dict(N=-1), dict(Hq=0), dict(Hkv=0), dict(Hq=2000), dict(D=96), dict(D=256),
                                    dict(qkv_dtype=3), dict(ld_qkv=767), dict(ld_qkv=770), dict(qkv_dtype=1, ld_qkv=772),
                                    dict(ld_q=511), dict(ld_q=516), dict(eps=-1.0), dict(eps=float("nan")),
                                    dict(rope_theta=0.0), dict(rope_theta=float("inf")), dict(qkv=P + 4),
                                    dict(q_out=P + 8), dict(kpool=P + 2), dict(vpool=P + 8), dict(q_gamma=P + 2),
                                    dict(k_gamma=P + 8), dict(qkv=0), dict(positions=0), dict(slots=0), dict(vpool=0),
                                    dict(kscale=0), dict(vscale=0), dict(page_size=17), dict(page_size=512),
                                    dict(num_pages=0), dict(num_pages=1 << 28)])
def test_stores_refuse(L, change):  # noqa: F811
    refused(L, "mk_qk_norm_rope_e4m3", NORM8, L.MK_ERR_ARG, **change)


def test_stores_refuse_more_rows_than_a_launch_has_blocks_for(L):  # noqa: F811
    refused(L, "mk_qk_norm_rope_e4m3", NORM8, L.MK_ERR_LIMIT, N=2 ** 31 - 1)


@pytest.mark.parametrize("change", [dict(B=-1), dict(N=-1), dict(max_new=0), dict(Hq=7), dict(Hkv=0), dict(D=96),
                                    dict(Hq=258, Hkv=2), dict(ld_q=511), dict(ld_q=516), dict(ld_out=511),
                                    dict(page_size=8), dict(page_size=48), dict(num_pages=0), dict(num_pages=1 << 27),
                                    dict(max_pages=0), dict(max_pages=1 << 27), dict(scale=0.0),
                                    dict(scale=float("inf")), dict(q=P + 8), dict(kpool=P + 8), dict(out=P + 2),
                                    dict(workspace=P + 4), dict(q=0), dict(kpool=0), dict(vpool=0), dict(table=0),
                                    dict(cu=0), dict(ctx_len=0), dict(out=0), dict(workspace=0), dict(kscale=0),
                                    dict(vscale=0)])
def test_attention_refuses(L, change):  # noqa: F811
    refused(L, "mk_paged_attention_e4m3", ATTN8, L.MK_ERR_ARG, **change)


def test_attention_workspace_refuses(L):  # noqa: F811
    for args in ((0, 8, 2, 64), (1, 7, 2, 64), (1, 8, 2, 65), (1, 8, 0, 64), (1, 258, 2, 64)):
        with pytest.raises(L.MkError) as e:
            L.mk_paged_attention_e4m3_workspace(*args)
        assert e.value.code == L.MK_ERR_ARG


@pytest.mark.parametrize("page_size,max_pages", [(16, (1 << 27) - 1), (16, (1 << 27) - 15), (128, (1 << 24) - 1)])
def test_attention_refuses_tables_up_to_the_end_of_int32(L, page_size, max_pages):  # noqa: F811
    assert max_pages * page_size < 2 ** 31
    refused(L, "mk_paged_attention_e4m3", ATTN8, L.MK_ERR_ARG, page_size=page_size, max_pages=max_pages)


def test_pools_of_another_type_and_their_workspace_are_refused():
    from task_graph_interpreter_gb300 import paged
    for dtype in (torch.float8_e5m2, torch.uint8, torch.float16, torch.float32):
        with pytest.raises(ValueError, match="pools"):
            paged.attention_workspace(1, 8, 2, 64, dtype=dtype)


@pytest.mark.parametrize("change", [dict(N=-1), dict(V=0), dict(V=1 << 30), dict(top=-1), dict(top=33), dict(V=4, top=5),
                                    dict(logits_dtype=0), dict(logits_dtype=3), dict(ld=999), dict(ld=-1000),
                                    dict(logits=P + 2), dict(logits=P + 1, logits_dtype=1), dict(logits=0),
                                    dict(logprobs=0), dict(entropy=0), dict(top_ids=0), dict(top_logprobs=0)])
def test_log_probabilities_refuse(L, change):  # noqa: F811
    refused(L, "mk_token_logprobs", SCORE, L.MK_ERR_ARG, **change)


def test_log_probabilities_refuse_too_many_rows(L):  # noqa: F811
    refused(L, "mk_token_logprobs", SCORE, L.MK_ERR_LIMIT, N=2 ** 31 - 1)


def test_the_library_exports_the_operators_on_8_bit_pages(L):  # noqa: F811
    header = re.sub(r"/\*.*?\*/", "", (pathlib.Path(__file__).parents[1] / "include" / "mk.h").read_text(), flags=re.S)
    declared = set(re.findall(r"\b(mk_\w+)\s*\(", header))
    assert declared == set(L.EXPORTS) | set(L.EXPORTS_E4M3)
    assert all(hasattr(L.lib(), name) for name in L.EXPORTS_E4M3)


def test_tensors_on_the_cpu_are_refused(L):  # noqa: F811
    from task_graph_interpreter_gb300 import logprobs, paged
    with pytest.raises(ValueError, match="CUDA"):
        logprobs.token_logprobs(torch.zeros(2, 10), torch.zeros(2, dtype=torch.int32))
    pool = torch.zeros(2, 2, 16, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
    scale, i = torch.ones(2, 2), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        paged.qk_norm_rope(torch.zeros(1, 8 * 64), 4, 2, 64, i, i, pool, pool, kscale=scale, vscale=scale)
    with pytest.raises(ValueError, match="CUDA"):
        paged.attention(torch.zeros(1, 4, 64).bfloat16(), pool, pool, i[None], i, i, 1, kscale=scale, vscale=scale)


def test_an_8_bit_cache_on_the_cpu_has_scales():
    from task_graph_interpreter_gb300 import paged
    c = paged.PagedCache(2, 4, 16, 2, 64, 2, 2, 8, device="cpu", dtype=torch.float8_e4m3fn)
    assert [t.shape for t in c.kscale + c.vscale] == [(4, 2)] * 4 and c.kpool[0].dtype == torch.float8_e4m3fn
    c = paged.PagedCache(2, 4, 16, 2, 64, 2, 2, 8, device="cpu")
    assert c.kscale == [None, None] and c.vpool[1].dtype == torch.bfloat16
    with pytest.raises(ValueError, match="float16"):
        paged.PagedCache(1, 4, 16, 2, 64, 2, 2, 8, device="cpu", dtype=torch.float16)
