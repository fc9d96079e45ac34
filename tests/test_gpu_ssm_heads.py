"""The scan's backward where a block walks several heads: as many chunks and
groups as SMs, so that no group's heads are cut into runs.  The sequences are
copies of two, and the reference is taken of those.  Entry-wise bounds as in
test_gpu_ssm.py, and norms as in ssm_norms.py."""
import pytest
import torch

import ssm_norms as N
import ssm_ref as R
from test_gpu_ssm import F64, GRADS, NAMES, SCAN, cu_of, dev, make, rels

pytestmark = pytest.mark.gpu
CHUNK = {"bf16": 128, "fp32": 64}


def copies(lens, G, dk, dv, dtype):
    """How often `lens` is repeated: the most that does not go beyond the SMs
    (fp32 at dk = dv = 64: two blocks an SM), and over three quarters of them."""
    room = torch.cuda.get_device_properties(0).multi_processor_count * (2 if dtype == "fp32" and dk + dv == 128 else 1)
    slots = lambda n: (sum(lens) * n // CHUNK[dtype] + len(lens) * n) * G  # noqa: E731  (packed: an upper bound otherwise)
    n = max(i for i in range(1, room + 1) if slots(i) <= room)
    assert slots(n) > 0.75 * room
    return n


def check(lens, H, G, dk, dv, dtype, packed, save=True, scale=None):
    import gated_delta_rule_gdn2_b200 as g
    T, B = sum(lens), len(lens)
    x = make(B, T, H, G, dk, dv, dtype, lens=lens, seed=121 + H)
    if scale is not None:  # heads of uneven size
        x["dO"] = x["dO"] * scale[:, None]
        x["dS_T"] = x["dS_T"] * scale[:, None, None]
    if packed:
        n = copies(lens, G, dk, dv, dtype)
    else:
        assert len(set(lens)) == 1
        per = -(-lens[0] // CHUNK[dtype]) * G * B
        room = torch.cuda.get_device_properties(0).multi_processor_count * (2 if dtype == "fp32" and dk + dv == 128 else 1)
        n = room // per
        assert n * per > 0.75 * room
    d = dev(x, dtype)
    big = {m: None if t is None else t if m == "skip" else t.repeat(n, *[1] * (t.dim() - 1)) for m, t in d.items()}
    cu = cu_of(lens * n) if packed else None
    if not packed:
        for m in ("q", "k", "v", "la", "dt", "dO"):
            big[m] = big[m].unflatten(0, (B * n, lens[0]))
    # (no room for partial sums of dq and dk: every block walks all the heads of its group)
    slots = sum(lens) * n // CHUNK[dtype] + B * n if packed else B * n * -(-lens[0] // CHUNK[dtype])
    up = lambda b: -(-b // 256) * 256  # noqa: E731
    code = g.GDN2_BF16 if dtype == "bf16" else g.GDN2_FP32
    sizes = (B * n, T * n if packed else lens[0], H, G, dk, dv, code, packed)
    size = g.gdn2_ssm_bwd_workspace(*sizes, 1) - g.gdn2_ssm_fwd_workspace(*sizes)  # (without the sequences' parts)
    images = up(slots * H * dk * dv * (2 if dtype == "bf16" else 4))
    assert size < images + up(4 * slots * H) + 2 * 4 * n * T * G * dk
    a = [big[m] for m in ("q", "k", "v", "la", "dt")]
    o, ST, st = g.ssm_fwd(*a, skip=big["skip"], S0=big["S0"], save_states=True, cu_seqlens=cu)
    gr = g.ssm_bwd(*a, big["dO"], skip=big["skip"], S0=big["S0"], dS_T=big["dS_T"], states=st if save else None, cu_seqlens=cu)
    assert g.gdn2_get_device_status() == 0
    y = {m: None if t is None else t.cuda() for m, t in x.items()}
    args = [y[m] for m in NAMES] + [y["dO"], y["dS_T"], lens]
    ref, mag = R.scan_grads(*args), R.magnitudes(*args)
    tok, f32 = rels(dtype, max(lens), dk, dv, 3)
    norm = N.BF16 if dtype == "bf16" else N.FP32
    for m in GRADS:
        got = gr[m].flatten(0, 1) if not packed else gr[m]
        got = got.unflatten(0, (n, T))
        assert torch.equal(got, got[:1].expand_as(got)), m  # (copies: wherever they lie)
        N.close(m, got[0], ref[m], norm, 1)
        R.within(m, got[0].to(F64).cpu(), ref[m].cpu(), mag[m].cpu(), *tok, mag["dla_sum"].cpu() if m == "dlog_alpha" else 0.0)
    N.close("dS0", gr["dS0"][:B], ref["dS0"], N.PARTS if dtype == "bf16" else N.FP32, 1)
    N.close("dskip", gr["dskip"][None], n * ref["dskip"][None], N.FP32, 0)  # (a number a head: over the heads together)
    return o, ST


@pytest.mark.parametrize("dtype", SCAN)
@pytest.mark.parametrize("T,H,G,dk,dv", [(100, 3, 1, 128, 64), (128, 16, 1, 128, 128), (60, 16, 1, 64, 64), (130, 6, 2, 64, 128),
                                         (100, 16, 1, 128, 64), (200, 5, 1, 128, 128)])
def test_every_head_of_a_block(T, H, G, dk, dv, dtype):
    check((T, T), H, G, dk, dv, dtype, False)


@pytest.mark.parametrize("dtype", SCAN)
@pytest.mark.parametrize("lens,H,G,dk,dv", [((90, 150), 16, 1, 128, 64), ((90, 150), 5, 1, 128, 128), ((256, 77), 3, 1, 64, 64),
                                            ((129, 64), 6, 2, 64, 128)])
def test_every_head_of_a_packed_block(lens, H, G, dk, dv, dtype):
    check(lens, H, G, dk, dv, dtype, True, save=H != 5)


@pytest.mark.parametrize("dtype", SCAN)
@pytest.mark.parametrize("lens,H,dk,dv", [((100, 100), 3, 128, 128), ((200, 200), 4, 64, 64), ((90, 150), 3, 128, 64)])
def test_a_large_head_leaves_the_others_digits(lens, H, dk, dv, dtype):
    """A head whose gradients are 2^20 times the others': theirs are as near as
    without it, whichever head of the block it is."""
    for at in (0, H - 1):
        scale = torch.ones(H, dtype=F64)
        scale[at] = 2.0 ** 20
        check(lens, H, 1, dk, dv, dtype, lens[0] != lens[1], scale=scale)
