"""The cache's calls have no backward pass: tensors that want one are refused instead of
silently cut off."""
import pytest
import torch

import speculative_decoding_rejection_02_gb300 as sv
from speculative_decoding_rejection_02_gb300 import _build


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()


def calls(device):
    pages = torch.zeros((2, 16, 1, 64), dtype=torch.bfloat16, device=device)
    x = torch.zeros((3, 1, 64), dtype=torch.bfloat16, device=device)
    i = torch.zeros(3, dtype=torch.int32, device=device)
    attend = dict(q=x, k_pages=pages, v_pages=pages.clone(), kv_lens=i[:1],
                  block_table=i[:1].view(1, 1), cu_q=i[:2], out=x.clone())
    append = dict(k=x, v=x.clone(), k_pages=pages, v_pages=pages.clone(),
                  slots=torch.zeros(3, dtype=torch.int64, device=device))
    return [(sv.cache_attend, attend, n) for n in ("q", "k_pages", "v_pages", "out")] + [
        (sv.cache_append, append, n) for n in ("k", "v", "k_pages", "v_pages")]


@pytest.mark.parametrize("which", [0, 4])  # the first argument, checked before its device
def test_refused(which):
    fn, kw, name = calls("cpu")[which]
    kw[name] = kw[name].requires_grad_()
    with pytest.raises(ValueError, match=f"{name} .*gradient"):
        fn(**kw)
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA device"):
        fn(**kw)


@pytest.mark.gpu
@pytest.mark.parametrize("which", range(8))
def test_accepted_without_gradients(which):
    fn, kw, name = calls("cuda:0")[which]
    kw[name] = kw[name].requires_grad_()
    with pytest.raises(ValueError, match=f"{name} .*gradient"):
        fn(**kw)
    with torch.no_grad():
        fn(**kw)
    with torch.inference_mode():
        fn(**kw)
    fn(**dict(kw, **{name: kw[name].detach()}))
