"""Which positions, frequencies and axes the calls with positions of several axes take: host checks (no GPU), and a call."""
import pytest
import torch

import exact_io_aware_06_gb300 as fa
from exact_io_aware_06_gb300._layer import _axes


def test_no_pairs_need_no_positions():
    # as fa_qk_norm_rope: without pairs nothing is turned, whether there are no frequencies or none of them
    f, axis = fa.rope_axes([0, 0])
    assert f.numel() == 0 and axis.numel() == 0
    for args in ((None, None, None), (None, f, axis), (None, f, None)):
        assert _axes(*args) == (1, None)
    assert _axes(torch.zeros((3, 1, 4), dtype=torch.int32), f, None) == (3, None)


def test_pairs_need_positions_and_axes():
    f, axis = fa.rope_axes([8, 8])
    pos = torch.zeros((2, 1, 4), dtype=torch.int32)
    assert _axes(pos, f, axis) == (2, axis.data_ptr())
    for args in ((None, f, axis), (pos[0], f, axis), (pos, f, None), (pos, f, axis.long()), (pos, f, axis[:7])):
        with pytest.raises(ValueError):
            _axes(*args)


@pytest.mark.gpu
def test_calls_without_pairs():
    import test_gpu_norm_rope as nr
    from gpu_util import check_status, ensure_built
    ensure_built()
    qkv, qw, kw, up = nr.make(2, 9, 4, 2, 64, "f32")
    f, axis = fa.rope_axes([0, 0, 0])
    out, out2 = (nr.outputs(2, 9, 4, 2, 64, torch.float32) for _ in range(2))
    fa.fa_qk_norm_rope_axes(qkv, qw, kw, None, f, axis, *out, 1e-6)
    fa.fa_qk_norm_rope(qkv, qw, kw, None, f, *out2, 1e-6)
    grads = [torch.empty_like(qkv) for _ in range(2)]
    fa.fa_qk_norm_rope_axes_bwd(qkv, qw, kw, None, f, axis, *up, grads[0], None, None, None, 1e-6)
    fa.fa_qk_norm_rope_bwd(qkv, qw, kw, None, f, *up, grads[1], None, None, None, 1e-6)
    check_status()
    for a, b in zip([*out, grads[0]], [*out2, grads[1]]):
        assert torch.equal(a, b)
