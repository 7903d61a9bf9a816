"""The binding of the adapters and norms given things that are no tensors, or tensors of other dimensions: a ValueError
that names the argument, as for a wrong type or shape."""
import numpy as np
import pytest
import torch

import group_wise_affine_qlinear_b200 as ql
from group_wise_affine_qlinear_b200 import build as qb

NOT_TENSORS = [None, 1.0, [1, 2], np.zeros((4, 256), np.float32), torch.tensor(1.0)]


def _args(dev):
    M, K, N, n, r = 4, 256, 64, 2, 8
    w = dict(codes=torch.zeros((N, K // 8), dtype=torch.int32, device=dev),
             scales=torch.zeros((N, K // 64), dtype=torch.float16, device=dev),
             biases=torch.zeros((N, K // 64), dtype=torch.float16, device=dev))
    return dict(x=torch.zeros((M, K), dtype=torch.bfloat16, device=dev), **w,
                lora_a=torch.zeros((n, r, K), dtype=torch.bfloat16, device=dev),
                lora_b=torch.zeros((n, N, r), dtype=torch.bfloat16, device=dev),
                adapter_ids=torch.zeros(M, dtype=torch.int32, device=dev))


def _check(dev, names):
    qb.build()
    good = _args(dev)
    for name in names:
        for bad in NOT_TENSORS + ([good[name][None]] if name in good else []):
            if bad is None and name in ("lora_scale", "out", "workspace"):
                continue                               # absent
            with pytest.raises(ValueError, match=name):
                ql.forward_lora(**{**good, name: bad})
    w = [good[k] for k in ("codes", "scales", "biases")]
    ad = [good["lora_a"], good["lora_b"]]
    for name in names:
        for bad in NOT_TENSORS:
            if name in ("lora_scale", "out", "workspace"):
                continue
            gate, up, gl, ul = list(w), list(w), list(ad), list(ad)
            x, ids = good["x"], good["adapter_ids"]
            if name == "x":
                x = bad
            elif name == "adapter_ids":
                ids = bad
            elif name in ("lora_a", "lora_b"):
                gl[name == "lora_b"] = bad
            else:
                gate[("codes", "scales", "biases").index(name)] = bad
            with pytest.raises(ValueError, match=name if name != "codes" else "gate codes"):
                ql.swiglu_lora(x, gate, up, gl, ul, ids)


def test_what_is_no_tensor_is_refused_by_name():
    _check("cpu", ["x", "codes", "lora_a", "lora_b"])
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    for bad in NOT_TENSORS:
        with pytest.raises(ValueError, match="x must be"):
            ql.norm_residual(bad)
        if bad is not None:
            with pytest.raises(ValueError, match="y must be"):
                ql.norm_residual(x, bad)
            for name in ("gate", "scale", "shift", "post_weight", "pre_weight"):
                with pytest.raises(ValueError, match=name):
                    ql.norm_residual(x, x, **{name: bad})


@pytest.mark.gpu
def test_what_is_no_tensor_is_refused_by_name_on_the_device():
    if not torch.cuda.is_available():
        pytest.fail("CUDA GPU required for -m gpu tests")
    _check("cuda", ["x", "codes", "scales", "biases", "lora_a", "lora_b", "adapter_ids", "lora_scale", "out", "workspace"])
    x = torch.zeros((4, 256), dtype=torch.bfloat16, device="cuda")
    for bad in NOT_TENSORS[1:]:
        for name in ("gate", "scale", "shift", "post_weight", "pre_weight", "segment_ids", "out", "h"):
            with pytest.raises(ValueError, match=name):
                ql.norm_residual(x, x, **{name: bad})
    assert ql.device_status() == 0
