"""Where the gradients of strided views are put: host code only."""
import pytest
import torch


def slices(w, H, G, dk, dv):
    return [w[..., H * dv + G * dk:H * dv + 2 * G * dk].unflatten(-1, (G, dk)), w[..., H * dv:H * dv + G * dk].unflatten(-1, (G, dk)),
            w[..., :H * dv].unflatten(-1, (H, dv))]


@pytest.mark.parametrize("lead", [(2, 50), (100,), (1, 50), (50, 1)])
def test_gradients_of_slices_share_one_tensor(lead):
    """Where q, k, v are slices of one tensor's rows, their gradients take no
    more than that tensor together, and no two overlap; otherwise each stands alone."""
    from gated_delta_rule_gdn2_b200.binding import _like_rows, _row_ld
    H, G, dk, dv = 4, 2, 64, 128

    def made(ts):
        lds = [_row_ld("t", t, len(lead), t.shape[-2] * t.shape[-1]) for t in ts]
        out = _like_rows(ts, lds)
        for i, (t, o) in enumerate(zip(ts, out)):
            assert o.shape == t.shape and o.dtype == t.dtype
            assert _row_ld("o", o, len(lead), t.shape[-2] * t.shape[-1]) == lds[i]
            o.fill_(i + 1)
        for i, o in enumerate(out):
            assert bool((o == i + 1).all())
        return sum({o.untyped_storage().data_ptr(): o.untyped_storage().nbytes() for o in out}.values())

    rows = 1
    for n in lead:
        rows *= n
    wide = torch.zeros(*lead, H * dv + 2 * G * dk + 40)  # (the rows end in something else)
    size = 4 * rows * (H * dv + 2 * G * dk)
    q, k, v = slices(wide, H, G, dk, dv)
    assert made([q, k, v]) <= size + 4 * rows * 40
    assert made([q.contiguous(), k.contiguous(), v.contiguous()]) == size
    assert made([q, k, v.contiguous()]) <= size + 4 * rows * (H * dv + 40)
    made([q, q, v])  # the same slice twice: gradients of their own
    made([q, k, slices(wide.clone(), H, G, dk, dv)[2]])
    made([k, q[..., ::1, :], v])
