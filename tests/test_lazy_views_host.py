"""A lazily conjugated or negated view has other values than its memory.  The calls read
memory, so such an argument is refused, before anything else about it is looked at."""
import pytest
import torch

from split_kv_mla_gb300 import mla


def args():
    z, i32 = torch.zeros, torch.int32
    ws = z(1 << 18, dtype=torch.uint8)
    i = z(4, dtype=i32)
    return {
        "reorder": (mla.mla_beam_reorder, dict(state=z(4, 10), parents=i, lens=i, tokens=i,
                                               out=z(4, 10), out_lens=i, workspace_t=ws)),
        "select": (mla.mla_beam_select, dict(logits=z(4, 10), scores=z(1, 4), tokens=i, parents=i,
                                             scores_out=z(1, 4), workspace_t=ws)),
        "extend": (mla.mla_cache_extend, dict(
            kv_indices=i, kv_indptr=z(5, dtype=i32), seq_lens=i, cursor=z(1, dtype=i32), total=8,
            num_tokens=4, pool_rows=100, workspace_t=ws)),
        "append": (mla.mla_cache_append, dict(
            kv=z(4, 576, dtype=torch.bfloat16), slots=i, pool=z(9, 576, dtype=torch.uint8),
            positions=i, cos_sin=z(9, 64), kv_scale=1.0, workspace_t=ws)),
    }


@pytest.mark.parametrize("call,name", [(c, n) for c, (_, kw) in args().items()
                                       for n, t in kw.items() if torch.is_tensor(t)])
def test_negated(call, name):
    f, kw = args()[call]
    kw[name] = torch._neg_view(kw[name])
    with pytest.raises(ValueError, match="lazily"):
        f(**kw)
    kw[name] = kw[name].resolve_neg()
    with pytest.raises(ValueError, match="CUDA|cuda"):    # the next thing that is wrong
        f(**kw)


@pytest.mark.parametrize("name", ["state", "out"])
def test_conjugated(name):
    f, kw = args()["reorder"]
    kw.update(state=torch.zeros(4, 10, dtype=torch.complex64), tokens=None,
              out=torch.zeros(4, 10, dtype=torch.complex64))
    kw[name] = kw[name].conj()
    with pytest.raises(ValueError, match="lazily"):
        f(**kw)
    # the imaginary part of one is a negated view
    f, kw = args()["reorder"]
    kw["state"] = torch.zeros(4, 10, dtype=torch.complex64).conj().imag
    with pytest.raises(ValueError, match="lazily"):
        f(**kw)


@pytest.mark.gpu
def test_resolved_complex_states():
    g = torch.Generator(device="cuda").manual_seed(1)
    state = torch.randn(5, 33, dtype=torch.complex64, generator=g, device="cuda").conj()
    parents = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="lazily"):
        mla.mla_beam_reorder(state, parents)
    out, _ = mla.mla_beam_reorder(state.resolve_conj(), parents)
    assert torch.equal(out, state[parents.long()]) and not out.is_conj()
