"""clip_grad_norm refuses lists in which one tensor's output overlaps another tensor, or its own gradient in part."""
import ctypes

import pytest
import torch

import row_wise_online_gb300 as rwo
from row_wise_online_gb300 import _build, train

X = 0x10000  # never dereferenced: what is not refused for its overlaps is for its workspace, or for want of a GPU


@pytest.fixture(scope="module", autouse=True)
def _built():
    _build.build()


def clip(*entries):
    arr = (train._Grad * len(entries))(*[train._Grad(*e) for e in entries])
    p = ctypes.cast(arr, ctypes.c_void_p)
    return rwo.capi().clip_grad_norm(p, len(entries), 1.0, 1.0, X, X + 128, 2 ** 40, None)


def apart(st):
    return st in (rwo.ERR_MISALIGNED, rwo.ERR_CUDA)


def test_lists():
    f, b = 0, 1  # fp32, bf16
    a = (X, X, 16, f, f)  # 64 bytes
    assert apart(clip(a)) and apart(clip(a, (X + 64, X + 64, 4, f, f))) and apart(clip((X + 64, X + 64, 4, f, f), a))
    assert clip(a, (X + 60, X + 60, 4, f, f)) == rwo.ERR_INVALID_ARG and clip((X + 60, X + 60, 4, f, f), a) == rwo.ERR_INVALID_ARG
    assert clip(a, (X + 8, X + 8, 2, f, f)) == rwo.ERR_INVALID_ARG and clip(a, a) == rwo.ERR_INVALID_ARG  # one inside the other
    assert apart(clip(a, (X + 8, X + 8, 0, f, f), (X, X, 0, f, f)))  # empty ones are nowhere
    # outputs
    assert apart(clip((X, X + 64, 16, f, f), (X + 128, X + 192, 16, f, f)))
    assert clip((X, X + 60, 16, f, f)) == rwo.ERR_INVALID_ARG and clip((X + 60, X, 16, f, f)) == rwo.ERR_INVALID_ARG  # over a part of its own gradient
    assert clip((X, X + 128, 16, f, f), (X + 128, X, 16, f, f)) == rwo.ERR_INVALID_ARG  # each where the other is read
    assert clip((X, X + 128, 16, f, f), (X + 64, X + 188, 16, f, f)) == rwo.ERR_INVALID_ARG
    assert clip((X, X + 64, 16, b, f), (X + 32, X + 256, 16, b, f), (X + 1024, X + 124, 4, b, f)) == rwo.ERR_INVALID_ARG  # fp32 ends later
    assert apart(clip((X, X + 64, 16, b, f), (X + 32, X + 256, 16, b, f), (X + 1024, X + 128, 4, b, f)))
    assert clip((X, X + 32, 16, b, b), (X + 512, X + 528, 16, b, b)) == rwo.ERR_INVALID_ARG and apart(clip((X, X + 32, 16, b, b), (X + 512, X + 544, 16, b, b)))
    # a gradient read twice is no overlap
    assert apart(clip((X, X + 64, 16, f, f), (X, X + 128, 16, f, f)))
    # long lists
    many = [(X + 64 * k, X + 64 * k, 16, f, f) for k in range(1000)]
    assert apart(clip(*many)) and apart(clip(*many[::-1]))
    assert clip(*many, (X + 64 * 500 + 60, X + 64 * 500 + 60, 1, f, f)) == rwo.ERR_INVALID_ARG


@pytest.mark.gpu
def test_views():
    torch.cuda.set_device(0)
    flat = torch.randn(4096, device="cuda")
    keep = flat.clone()
    a, b = flat[:1024], flat[1024:2048]
    for call in (lambda: rwo.clip_grad_norm([flat, flat[5:9]], 1e-3), lambda: rwo.clip_grad_norm([a, flat[1000:1100]], 1e-3),
                 lambda: rwo.clip_grad_norm([a, b], 1e-3, out=[b, a]), lambda: rwo.clip_grad_norm([a], 1e-3, out=[flat[4:1028]])):
        with pytest.raises(rwo.SoftmaxError):
            call()
    torch.cuda.synchronize()
    assert torch.equal(flat, keep)
    out = [torch.empty_like(a), torch.empty_like(a)]
    rwo.clip_grad_norm([a, a], 1e-3, out=out)  # read twice
    assert torch.equal(out[0], out[1]) and rwo.get_status() == rwo.OK
    rwo.clip_grad_norm([b, a], 1e-3)  # neighbours
    assert rwo.get_status() == rwo.OK and not torch.equal(a, keep[:1024])
