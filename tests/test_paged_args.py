"""Refusals of the paged-cache operators and of draft verification (no GPU:
what the host checks is refused before any device work, so fake aligned
addresses stand in for device memory)."""
import pytest
import torch

P = 1 << 20  # an aligned address nothing reads


@pytest.fixture(scope="module")
def L():
    from task_graph_interpreter_gb300 import build as _b
    _b()
    from task_graph_interpreter_gb300 import _lib
    _lib.lib()
    return _lib


PLAN = dict(stream=0, B=4, page_size=16, max_pages=8, num_pages=64, max_tokens=32, ctx_len=P, new_len=P, table=P,
            held=P, held_out=P, free_pages=P, free_count=P, free_count_out=P, cu=P, positions=P, slots=P)
NORM = dict(stream=0, N=4, Hq=8, Hkv=2, D=64, qkv=P, qkv_dtype=2, ld_qkv=768, q_gamma=0, k_gamma=0, eps=1e-5,
            rope_theta=5e5, positions=P, slots=P, q_out=P, ld_q=512, kpool=P, vpool=P, num_pages=64, page_size=16)
ATTN = dict(stream=0, B=2, N=4, max_new=4, Hq=8, Hkv=2, D=64, q=P, ld_q=512, kpool=P, vpool=P, num_pages=64,
            page_size=16, table=P, max_pages=8, cu=P, ctx_len=P, scale=0.125, out=P, ld_out=512, workspace=P,
            workspace_size=1 << 30)
VERIFY = dict(stream=0, B=2, K=4, V=1000, p=P, ld_p=1000, q=P, ld_q=1000, drafts=P, draft_len=0, u=P, tokens=P,
              accepted=P)


def refused(L, fn, base, code, **change):
    with pytest.raises(L.MkError) as e:
        getattr(L, fn)(**{**base, **change})
    assert e.value.code == code, str(e.value)
    assert fn in str(e.value)


@pytest.mark.parametrize("change", [dict(B=0), dict(B=4097), dict(page_size=0), dict(page_size=24), dict(page_size=512),
                                    dict(page_size=8), dict(max_pages=0), dict(num_pages=0), dict(max_tokens=0),
                                    dict(ctx_len=0), dict(new_len=0), dict(table=0), dict(held=0), dict(held_out=0),
                                    dict(free_pages=0), dict(free_count=0), dict(free_count_out=0), dict(cu=0),
                                    dict(positions=0), dict(slots=0)])
def test_plan_refuses(L, change):
    refused(L, "mk_paged_plan", PLAN, L.MK_ERR_ARG, **change)


@pytest.mark.parametrize("change", [dict(num_pages=1 << 28), dict(max_pages=1 << 28), dict(max_tokens=2 ** 31 - 1)])
def test_plan_refuses_what_int32_does_not_hold(L, change):
    refused(L, "mk_paged_plan", PLAN, L.MK_ERR_LIMIT, **change)


@pytest.mark.parametrize("change", [dict(N=-1), dict(Hq=0), dict(Hkv=0), dict(Hq=2000), dict(D=96), dict(D=256),
                                    dict(qkv_dtype=3), dict(ld_qkv=767), dict(ld_qkv=770), dict(qkv_dtype=1, ld_qkv=772),
                                    dict(ld_q=511), dict(ld_q=516), dict(eps=-1.0), dict(eps=float("nan")),
                                    dict(rope_theta=0.0), dict(rope_theta=float("inf")), dict(qkv=P + 4),
                                    dict(q_out=P + 8), dict(kpool=P + 2), dict(q_gamma=P + 2), dict(k_gamma=P + 8),
                                    dict(qkv=0), dict(positions=0), dict(slots=0), dict(vpool=0), dict(page_size=17),
                                    dict(num_pages=0), dict(num_pages=1 << 28)])
def test_norm_rope_refuses(L, change):
    refused(L, "mk_qk_norm_rope", NORM, L.MK_ERR_ARG, **change)


@pytest.mark.parametrize("change", [dict(B=-1), dict(N=-1), dict(max_new=0), dict(Hq=7), dict(Hq=1), dict(Hkv=0),
                                    dict(Hq=258, Hkv=2, ld_q=1 << 15, ld_out=1 << 15), dict(D=80), dict(page_size=20),
                                    dict(num_pages=0), dict(num_pages=1 << 27), dict(max_pages=0), dict(ld_q=504),
                                    dict(ld_q=516), dict(ld_out=504), dict(ld_out=513), dict(scale=0.0),
                                    dict(scale=float("nan")), dict(scale=-1.0), dict(q=0), dict(q=P + 8), dict(out=P + 4),
                                    dict(kpool=P + 8), dict(vpool=0), dict(table=0), dict(cu=0), dict(ctx_len=0),
                                    dict(workspace=0), dict(workspace=P + 4)])
def test_attention_refuses(L, change):
    refused(L, "mk_paged_attention", ATTN, L.MK_ERR_ARG, **change)


def test_attention_workspace_refuses(L):
    for args in ((0, 8, 2, 64), (1, 7, 2, 64), (1, 8, 2, 65), (1, 8, 0, 64)):
        with pytest.raises(L.MkError) as e:
            L.mk_paged_attention_workspace(*args)
        assert e.value.code == L.MK_ERR_ARG


@pytest.mark.parametrize("change", [dict(B=-1), dict(K=-1), dict(K=1025), dict(V=0), dict(ld_p=999), dict(ld_q=999),
                                    dict(p=0), dict(u=0), dict(drafts=0), dict(tokens=0), dict(accepted=0)])
def test_verify_refuses(L, change):
    refused(L, "mk_verify_drafts", VERIFY, L.MK_ERR_ARG, **change)


@pytest.mark.parametrize("change", [dict(V=(1 << 28) + 1, ld_p=1 << 29, ld_q=1 << 29), dict(B=(1 << 24) + 1)])
def test_verify_refuses_what_is_too_large(L, change):
    refused(L, "mk_verify_drafts", VERIFY, L.MK_ERR_LIMIT, **change)


def test_tensor_functions_refuse_host_tensors():
    from task_graph_interpreter_gb300 import paged, speculative
    i = torch.zeros(4, dtype=torch.int32)
    pool = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        paged.plan(i, i, i.view(2, 2), i, i, i, 16, max_tokens=4)
    with pytest.raises(ValueError):
        paged.qk_norm_rope(torch.zeros(4, 256), 2, 1, 64, i, i, pool, pool)
    with pytest.raises(ValueError):
        paged.attention(torch.zeros(4, 2, 64, dtype=torch.bfloat16), pool, pool, i.view(2, 2), i, i[:2], 1)
    with pytest.raises(ValueError):
        speculative.verify_drafts(torch.zeros(2, 3, 10), i.view(2, 2), torch.zeros(2, 3))


@pytest.mark.parametrize("page_size,max_pages", [(16, (1 << 27) - 1), (16, (1 << 27) - 15), (128, (1 << 24) - 1)])
def test_attention_refuses_tables_up_to_the_end_of_int32(L, page_size, max_pages):
    """The kernels count keys in whole blocks of up to 128, and rows of a tile up to 254 past a request's last: the
    last 255 positions that int32 holds are theirs."""
    assert max_pages * page_size < 2 ** 31
    refused(L, "mk_paged_attention", ATTN, L.MK_ERR_ARG, page_size=page_size, max_pages=max_pages)
