"""GPU: the new outputs of a call are tensors like others: each has its own memory, grows
without touching the others and keeps none of theirs."""
import pytest
import torch

from split_kv_mla_gb300 import mla

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    mla.load()


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def select(batch=3, K=4):
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(batch * 4, 300, generator=g, device="cuda")
    return mla.mla_beam_select(x, torch.zeros(batch, 4, device="cuda"), K, end_token=3)


def extend(requests=3, tokens=2):
    ptr = (torch.arange(requests + 1, device="cuda") * 5).int()
    lens = torch.full((requests,), 5, dtype=torch.int32, device="cuda")
    new = torch.full((requests,), tokens, dtype=torch.int32, device="cuda")
    n = 5 * requests
    return mla.mla_cache_extend(torch.arange(n, device="cuda").int(), ptr, lens, i32(n),
                                n + tokens * requests, tokens * requests, 1 << 30, new_tokens=new)


def reorder():
    return mla.mla_beam_reorder(torch.arange(40, device="cuda").int().view(4, 10), i32(3, 0, 1),
                                i32(5, 6, 7, 8))


@pytest.mark.parametrize("call", [select, extend, reorder])
def test_none_grows_over_another(call):
    want = [t.clone() for t in call()]
    for k in range(len(want)):
        for n in (want[k].numel() + 1, want[k].numel() + 8, 4000):
            out = call()
            out[k].resize_(n).fill_(7)
            for j, t in enumerate(out):
                assert j == k or torch.equal(t, want[j]), (j, k)


@pytest.mark.parametrize("call", [select, extend, reorder])
def test_they_are_tensors_like_others(call):
    for t in call():
        u = t.clone().resize_(t.numel() + 5)
        assert u.numel() == t.numel() + 5
        v = t.view(-1)[1:].reshape(-1, 1).unsqueeze(0)
        assert v.numel() == t.numel() - 1
        t += t.to(t.dtype) if t.dtype != torch.bool else t.logical_not()
        t.copy_(t.clone()), t.zero_()
        assert not t.any() and t.is_contiguous() and not t.requires_grad


def test_none_keeps_another():
    for out in (select(), select(3000, 16), extend(), extend(4, 300000), extend(0), reorder()):
        at = [t.untyped_storage().data_ptr() for t in out if t.numel()]
        assert len(set(at)) == len(at)
        for t in out:
            assert t.untyped_storage().nbytes() == t.numel() * t.element_size()
            assert t.storage_offset() == 0 and t.data_ptr() % 16 == 0
