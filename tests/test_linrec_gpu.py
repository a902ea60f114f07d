"""Gated linear recurrence (ssm_linrec_fwd, ssm_linrec_bwd) against the plain
64-bit recurrence on the same inputs.

Tolerances, derived: a gate carries about 4 fp32 roundings (2.4e-7) and the state
remembers about 1 / (1 - a) steps; with gates around sigmoid(2) a channel's
memory stays below about 20 steps, so an fp32 output is within 20 * 2.4e-7 = 5e-6,
taken as 1e-5, of the tensor's largest value, and a gradient, which multiplies
two such quantities, within 2e-5.  A bf16 output adds half an ulp, 2^-8 of the
value."""
import numpy as np
import pytest
import torch

from state_space_model_selective_gb300 import binding
from tests import plain64 as P
from tests.helpers import to64

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
OK, TIMEOUT = 0, 7
UNWRITTEN = -7.25e33


def _near(got, ref, what, tol):
    bf16 = got.dtype == BF16
    got = to64(got)
    assert got.shape == ref.shape, what
    if ref.size == 0:
        return
    # what is not finite in the reference (an infinite input that a step took) has to
    # be the same here
    fine = np.isfinite(ref)
    np.testing.assert_array_equal(got[~fine], ref[~fine], err_msg=what)
    got, ref = got[fine], ref[fine]
    assert np.all(np.isfinite(got)), what
    lim = tol * np.max(np.abs(ref)) + (2.0 ** -8 * np.abs(ref) * (1 + 1e-3) if bf16 else 0.0)
    bad = np.abs(got - ref) > lim
    assert not bad.any(), (what, float(np.max(np.abs(got - ref))), int(bad.sum()))


def _inputs(batch, n, dim, dtype, seed, gated=True, state=True):
    g = torch.Generator().manual_seed(seed)

    def randn(*s):
        return torch.randn(*s, generator=g)

    f = (2 + 1.5 * randn(batch, n, dim)).to(dtype)
    x, z, dy = (randn(batch, n, dim).to(dtype) for _ in range(3))
    h0, dfin = randn(batch, dim), randn(batch, dim)
    return {"f": f, "x": x, "z": z if gated else None, "dy": dy,
            "h0": h0 if state else None, "dfin": dfin if state else None}


def _dev(d):
    return {k: None if v is None else v.cuda() for k, v in d.items()}


def _n64(d):
    return {k: None if v is None else to64(v) for k, v in d.items()}


def _check(d, dev=None, out_dtype=None, grad_dtype=None):
    """Forward with kept states, gradient from them and without them."""
    dev = dev or _dev(d)
    r = _n64(d)
    batch, n, dim = d["x"].shape
    kept = torch.full((binding.ssm_linrec_checkpoint_bytes(batch, n, dim) // 4,), UNWRITTEN,
                      device="cuda")
    y, fin = binding.ssm_linrec_fwd(dev["f"], dev["x"], dev["z"], initial_state=dev["h0"],
                                    checkpoints=kept, out_dtype=out_dtype)
    y_ref, fin_ref, _ = P.linrec_fwd(r["f"], r["x"], r["z"], r["h0"])
    _near(y, y_ref, "y", 1e-5)
    _near(fin, fin_ref, "final", 1e-5)
    assert not (kept == UNWRITTEN).any()
    refs = P.linrec_bwd(r["f"], r["x"], r["dy"], r["z"], r["h0"], r["dfin"])
    grads = []
    for c in (kept, None):
        g = binding.ssm_linrec_bwd(dev["f"], dev["x"], dev["dy"], dev["z"],
                                   initial_state=dev["h0"], dfinal_state=dev["dfin"],
                                   checkpoints=c, grad_dtype=grad_dtype)
        for k, ref in zip(("df", "dx", "dz", "dinitial_state"), refs):
            if ref is None:
                assert g[k] is None
            else:
                _near(g[k], ref, k, 2e-5)
        grads.append(g)
    for k in ("df", "dx", "dinitial_state"):  # the kept states are the ones taken again
        assert torch.equal(grads[0][k], grads[1][k]), k


# lengths around the walked 16 steps, the 64- and 128-step tiles and the 32 tiles
# of one look-back round; channels around the 64 of a tile, with rows of 16, 4 and
# 2-byte alignment
SIZES = [(1, 1, 1), (2, 1, 130), (1, 2, 64), (3, 16, 65), (2, 17, 64), (1, 63, 8), (1, 64, 66),
         (2, 65, 63), (1, 127, 128), (2, 128, 72), (1, 129, 40), (3, 300, 77), (1, 1021, 129),
         (1, 4200, 16), (2, 5000, 3), (5, 257, 192), (70, 90, 24)]


@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("gated,state", [(True, True), (False, False)])
def test_matches_plain(size, dtype, gated, state):
    _check(_inputs(*size, dtype, sum(size), gated, state))


@pytest.mark.parametrize("dtype,other", [(F32, BF16), (BF16, F32)])
def test_other_output_types(dtype, other):
    _check(_inputs(2, 150, 70, dtype, 9), out_dtype=other, grad_dtype=other)
    _check(_inputs(2, 9, 70, dtype, 9), out_dtype=other, grad_dtype=other)


@pytest.mark.parametrize("n", [1, 200])
@pytest.mark.parametrize("dim", [64, 66, 35])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_slices_of_one_projection(n, dim, dtype):
    """f, x and z as column ranges of one tensor, in two orders: at odd widths
    neither the rows nor the ranges' starts are aligned."""
    d = _inputs(2, n, dim, dtype, dim + n)
    for order in ("fxz", "zfx"):
        packed = torch.cat([d[k] for k in order], -1).cuda()
        dev = _dev(d)
        for i, k in enumerate(order):
            dev[k] = packed[..., i * dim:(i + 1) * dim]
        _check(d, dev)


@pytest.mark.parametrize("pad", [0, 1, 7])
@pytest.mark.parametrize("dtype,out", [(F32, F32), (BF16, BF16), (F32, BF16), (BF16, F32)])
def test_rows_that_move_against_alignment(pad, dtype, out):
    """Several tiles of several channel blocks in every direction, where inputs (ranges of
    a padded projection) and outputs step by different bytes against 16-byte boundaries."""
    for dim, gated in ((131, True), (201, False)):
        d = _inputs(2, 333, dim, dtype, dim + pad, gated)
        order = "fxz" if gated else "xf"
        packed = torch.cat([torch.zeros(2, 333, pad, dtype=dtype)] + [d[k] for k in order],
                           -1).cuda()
        dev = _dev(d)
        for i, k in enumerate(order):
            dev[k] = packed[..., pad + i * dim:pad + (i + 1) * dim]
        _check(d, dev, out, out)


@pytest.mark.parametrize("n", [12, 300])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_masked_steps(n, dtype):
    """Gates of +inf over NaN and infinite inputs (padding), gates of -inf and of the
    type's lowest value (a new sequence), whole rows and channels of each, and a
    state of NaN dropped at the first step."""
    d = _inputs(3, n, 70, dtype, n)
    low = torch.finfo(dtype).min
    d["f"][0, n // 2:] = float("inf")          # a ragged end
    d["x"][0, n // 2:] = float("nan")
    d["f"][1, :, 5] = float("inf")             # a channel that never takes input
    d["x"][1, :, 5] = float("-inf")
    d["f"][1, 3] = float("-inf")
    d["f"][1, 7, 1:9] = low
    d["f"][2, :, 11] = float("-inf")           # a channel without memory
    d["f"][2, 0] = float("-inf")
    d["h0"][2] = float("nan")
    d["h0"][2, 3] = float("inf")
    _check(d)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_nan_reaches_its_channel_only(dtype):
    d = _dev(_inputs(1, 200, 72, dtype, 4, state=False))
    clean, _ = binding.ssm_linrec_fwd(d["f"], d["x"])
    d["f"][0, 70, 9] = float("nan")
    y, fin = binding.ssm_linrec_fwd(d["f"], d["x"])
    assert y[0, 70:, 9].isnan().all() and fin[0, 9].isnan()
    rest = torch.ones_like(y, dtype=torch.bool)
    rest[0, 70:, 9] = False
    assert torch.equal(y[rest], clean[rest])


def test_empty_sequence_and_no_channels():
    h0 = torch.randn(3, 70, device="cuda")
    e = torch.empty(3, 0, 70, device="cuda")
    y, fin = binding.ssm_linrec_fwd(e, e, initial_state=h0)
    assert y.shape == (3, 0, 70) and torch.equal(fin, h0)
    _, fin = binding.ssm_linrec_fwd(e, e)
    assert not fin.any()
    g = binding.ssm_linrec_bwd(e, e, e, dfinal_state=h0)
    assert torch.equal(g["dinitial_state"], h0)
    assert not binding.ssm_linrec_bwd(e, e, e)["dinitial_state"].any()
    for shape in ((0, 5, 70), (2, 5, 0)):
        e = torch.empty(*shape, device="cuda")
        y, fin = binding.ssm_linrec_fwd(e, e)
        assert y.shape == shape and fin.shape == (shape[0], shape[2])


def test_decode_steps_continue_a_prefill():
    """A prefill, then single tokens with the state updated in place, against the
    whole sequence at once."""
    d = _dev(_inputs(4, 160, 134, F32, 8))
    whole, fin = binding.ssm_linrec_fwd(d["f"], d["x"], d["z"], initial_state=d["h0"])
    y, state = binding.ssm_linrec_fwd(d["f"][:, :150].contiguous(), d["x"][:, :150].contiguous(),
                                      d["z"][:, :150].contiguous(), initial_state=d["h0"])
    parts = [y]
    for t in range(150, 160):
        step = [d[k][:, t:t + 1].contiguous() for k in "fxz"]
        y, out = binding.ssm_linrec_fwd(*step, initial_state=state, final_state=state)
        assert out is state
        parts.append(y)
    _near(torch.cat(parts, 1), to64(whole), "y", 1e-6)
    _near(state, to64(fin), "final", 1e-6)


def test_pieces_cut_at_tiles_give_the_bits_of_the_whole():
    d = _dev(_inputs(2, 512, 100, BF16, 10, gated=False, state=False))
    whole, fin = binding.ssm_linrec_fwd(d["f"], d["x"])
    state, parts = None, []
    for a, b in ((0, 128), (128, 384), (384, 512)):
        y, state = binding.ssm_linrec_fwd(d["f"][:, a:b].contiguous(),
                                          d["x"][:, a:b].contiguous(), initial_state=state)
        parts.append(y)
    assert torch.equal(torch.cat(parts, 1), whole) and torch.equal(state, fin)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_many_tiles_are_bit_equal_run_to_run(dtype):
    """Few channels and many tiles: how far each look-back has to go depends on
    timing, its result does not."""
    d = _dev(_inputs(1, 20000, 128, dtype, 11))
    runs = []
    for _ in range(4):
        y, fin = binding.ssm_linrec_fwd(d["f"], d["x"], d["z"], initial_state=d["h0"])
        g = binding.ssm_linrec_bwd(d["f"], d["x"], d["dy"], d["z"], initial_state=d["h0"])
        runs.append((y, fin, g["df"], g["dx"], g["dz"], g["dinitial_state"]))
    for r in runs[1:]:
        assert all(torch.equal(u, v) for u, v in zip(r, runs[0]))
    c = {k: None if v is None else to64(v) for k, v in d.items()}
    _near(runs[0][0], P.linrec_fwd(c["f"], c["x"], c["z"], c["h0"])[0], "y", 1e-5)


def test_another_stream_than_the_tensors_own():
    d = _dev(_inputs(2, 700, 96, BF16, 12))
    y, fin = binding.ssm_linrec_fwd(d["f"], d["x"], d["z"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    runs = [binding.ssm_linrec_fwd(d["f"], d["x"], d["z"], stream=side) for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(r[0], y) and torch.equal(r[1], fin) for r in runs)


def test_capture_in_a_graph():
    d = _dev(_inputs(2, 300, 96, BF16, 13))
    y, fin = binding.ssm_linrec_fwd(d["f"], d["x"], d["z"])
    want = (y.clone(), fin.clone())
    ws = torch.empty(binding.ssm_linrec_workspace_bytes(2, 300, 96), dtype=torch.uint8,
                     device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.ssm_linrec_fwd(d["f"], d["x"], d["z"], y=y, final_state=fin, workspace=ws)
    for _ in range(3):
        y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[0]) and torch.equal(fin, want[1])
        assert binding.ssm_last_device_status(ws) == OK


@pytest.mark.parametrize("grad", [False, True])
def test_look_back_gives_up_and_reports(grad):
    """The first tile withholds its state: the wait runs out at its limit, the status
    says so, and the next call is whole again."""
    d = _dev(_inputs(1, 1000, 64, BF16, 14, state=False))
    fb, bb = (binding.ssm_linrec_workspace_bytes(1, 1000, 64),
              binding.ssm_linrec_bwd_workspace_bytes(1, 1000, 64))
    ws = torch.empty(max(fb, bb), dtype=torch.uint8, device="cuda")

    def call():
        if grad:
            return binding.ssm_linrec_bwd(d["f"], d["x"], d["dy"], workspace=ws)["df"]
        return binding.ssm_linrec_fwd(d["f"], d["x"], workspace=ws)[0]

    want = call()
    assert binding.ssm_last_device_status(ws) == OK
    try:
        binding.ssm_debug_set_lookback(True, 500)
        call()
        status = binding.ssm_last_device_status(ws)
    finally:
        binding.ssm_debug_set_lookback()
    assert status == TIMEOUT
    assert torch.equal(call(), want)
    assert binding.ssm_last_device_status(ws) == OK


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("n,dim", [(1, 67), (150, 67), (150, 64)])
def test_writes_stay_inside_the_outputs(n, dim, dtype):
    """Every output between guards that must survive, every input unchanged."""
    d = _dev(_inputs(2, n, dim, dtype, 15))
    before = {k: v.clone() for k, v in d.items()}

    def guarded(shape, dt):
        num = int(np.prod(shape))
        buf = torch.full((num + 128,), -7.25e33, dtype=dt, device="cuda")
        buf[64:64 + num] = float("nan")
        return buf, buf[64:64 + num].view(shape)

    act, st = (2, n, dim), (2, dim)
    kept = (binding.ssm_linrec_checkpoint_bytes(2, n, dim) // 4,)
    bufs = {"y": guarded(act, dtype), "final_state": guarded(st, F32),
            "checkpoints": guarded(kept, F32)}
    binding.ssm_linrec_fwd(d["f"], d["x"], d["z"], initial_state=d["h0"],
                           **{k: v[1] for k, v in bufs.items()})
    outs = {"df": guarded(act, dtype), "dx": guarded(act, dtype), "dz": guarded(act, dtype),
            "dinitial_state": guarded(st, F32)}
    binding.ssm_linrec_bwd(d["f"], d["x"], d["dy"], d["z"], initial_state=d["h0"],
                           dfinal_state=d["dfin"], checkpoints=bufs["checkpoints"][1],
                           out={k: v[1] for k, v in outs.items()})
    torch.cuda.synchronize()
    for k, (buf, t) in {**bufs, **outs}.items():
        guard = torch.full((64,), -7.25e33, dtype=buf.dtype, device="cuda")
        assert torch.equal(buf[:64], guard) and torch.equal(buf[-64:], guard), k
        assert not t.isnan().any(), k
    for k, v in before.items():
        assert torch.equal(d[k], v), k


@pytest.mark.parametrize("n", [12, 300, 1500])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_what_is_not_finite_outlasts_a_span_that_forgets(n, dtype):
    """Gates around sigmoid(-1.5), so that the product of a tile's gates lies below every
    fp32 number, but none that restarts the state: NaN and infinities in x, in the
    initial state, in dy and in dfinal_state stay to the sequence's end (or its start), as
    they do step by step; a restart behind one ends it."""
    for dim in (70, 64):
        d = _inputs(4, n, dim, dtype, n + dim)
        d["f"] = (-1.5 + 0.3 * (d["f"].float() - 2)).to(dtype)
        d["x"][0, 5, 3], d["x"][1, 6, 9], d["x"][1, 6, 10] = float("nan"), float("inf"), -float("inf")
        d["x"][0, 5, 40], d["f"][0, n // 2, 40] = float("nan"), float("-inf")
        d["h0"][2, 4], d["h0"][2, 5], d["h0"][2, 41] = float("inf"), float("nan"), -float("inf")
        d["f"][2, n // 2, 41] = float("-inf")
        d["dy"][3, n - 3, 20] = float("nan")
        d["dfin"][3, 7], d["dfin"][3, 8] = float("nan"), float("inf")
        dev, r = _dev(d), _n64(d)
        kept = torch.empty(binding.ssm_linrec_checkpoint_bytes(4, n, dim) // 4, device="cuda")
        y, fin = binding.ssm_linrec_fwd(dev["f"], dev["x"], dev["z"], initial_state=dev["h0"],
                                        checkpoints=kept)
        y_ref, fin_ref, _ = P.linrec_fwd(r["f"], r["x"], r["z"], r["h0"])
        assert np.isnan(fin_ref[0, 3]) and np.isfinite(fin_ref[0, 40]) and fin_ref[2, 4] == np.inf
        _near(fin, fin_ref, "final", 1e-5)
        _near(y, y_ref, "y", 1e-5)
        refs = P.linrec_bwd(r["f"], r["x"], r["dy"], r["z"], r["h0"], r["dfin"])
        assert np.isnan(refs[3][3, 7]) and refs[3][3, 8] == np.inf and np.isnan(refs[3][3, 20])
        for c in (kept, None):
            g = binding.ssm_linrec_bwd(dev["f"], dev["x"], dev["dy"], dev["z"],
                                       initial_state=dev["h0"], dfinal_state=dev["dfin"],
                                       checkpoints=c)
            for k, ref in zip(("df", "dx", "dz", "dinitial_state"), refs):
                _near(g[k], ref, k, 2e-5)


def test_more_than_two_to_the_26_channel_blocks():
    """Sequences of two tiles, so many that an entry's number in the work area passes 31
    bits: the last ones' states come from their own first tiles, forwards and backwards."""
    batch, n = 2 ** 26 + 64, 65
    need = binding.ssm_linrec_bwd_workspace_bytes(batch, n, 1)
    if torch.cuda.mem_get_info()[0] < need + 9 * batch * n * 2:
        pytest.skip("needs about 180 GB of device memory")
    g = torch.Generator(device="cuda").manual_seed(16)

    def randn(*shape, dtype=BF16):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)

    f = randn(batch, n, 1).mul_(1.5).add_(2)
    x, dy, h0 = randn(batch, n, 1), randn(batch, n, 1), randn(batch, 1, dtype=F32)
    kept = torch.empty(binding.ssm_linrec_checkpoint_bytes(batch, n, 1) // 4, device="cuda")
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    y, fin = binding.ssm_linrec_fwd(f, x, initial_state=h0, checkpoints=kept, workspace=ws)
    assert binding.ssm_last_device_status(ws) == OK
    grads = binding.ssm_linrec_bwd(f, x, dy, initial_state=h0, checkpoints=kept, workspace=ws)
    assert binding.ssm_last_device_status(ws) == OK
    for at in (slice(0, 40), slice(2 ** 25 - 20, 2 ** 25 + 20), slice(2 ** 26 - 40, batch)):
        c = [to64(t[at]) for t in (f, x, dy, h0)]
        y_ref, fin_ref, _ = P.linrec_fwd(c[0], c[1], None, c[3])
        _near(y[at], y_ref, "y", 1e-5)
        _near(fin[at], fin_ref, "final", 1e-5)
        refs = P.linrec_bwd(c[0], c[1], c[2], None, c[3])
        for k, ref in zip(("df", "dx", "dz", "dinitial_state"), refs):
            if ref is not None:
                _near(grads[k][at], ref, k, 2e-5)
    del f, x, dy, h0, kept, ws, y, fin, grads
    torch.cuda.empty_cache()


@pytest.mark.parametrize("n,dim", [(24, 262144), (300, 64), (9, 64)])
def test_a_gradient_can_report_whatever_forward_it_ran(n, dim):
    """A gradient without kept states runs its forward first (24 steps of many channels by
    the walk) and keeps its status.  What both leave is the word over which a wait that runs
    out is recorded, all ones, and it reads as OK."""
    d = _dev(_inputs(1, n, dim, BF16, 17, gated=False, state=False))
    ws = torch.zeros(binding.ssm_linrec_bwd_workspace_bytes(1, n, dim), dtype=torch.uint8,
                     device="cuda")
    binding.ssm_linrec_bwd(d["f"], d["x"], d["dy"], workspace=ws)
    assert binding.ssm_last_device_status(ws) == OK
    assert int(ws[:8].view(torch.int32)[1]) == -1


@pytest.mark.parametrize("n", [9, 24, 20000])
@pytest.mark.parametrize("dim", [8, 7])
def test_long_memory(n, dim):
    """Constant gates close to 1, a channel to each f.  A gate and each update carry fp32
    roundings of up to 2^-22 of the state, which a channel remembers for 1 / (1 - a) = 1 +
    e^f steps: the state is within 2^-22 min(1 + e^f, n), and 1 - a, whose exponent is rounded
    once, within (|f| + 8) 2^-24, of the channel's largest.  The gradients multiply two such
    quantities."""
    f0 = torch.tensor([2.0, 4.0, 6.0, 8.0, 10.0, 12.0, 14.0, 16.0][:dim])
    d = _inputs(2, n, dim, F32, n + dim, gated=False)
    d["f"], d["x"] = f0.expand(2, n, dim).contiguous(), 1 + d["x"]
    dev, r = _dev(d), _n64(d)
    y, fin = binding.ssm_linrec_fwd(dev["f"], dev["x"], initial_state=dev["h0"])
    g = binding.ssm_linrec_bwd(dev["f"], dev["x"], dev["dy"], initial_state=dev["h0"],
                               dfinal_state=dev["dfin"])
    y_ref, fin_ref, _ = P.linrec_fwd(r["f"], r["x"], None, r["h0"])
    df, dx, _, dh0 = P.linrec_bwd(r["f"], r["x"], r["dy"], None, r["h0"], r["dfin"])
    for c in range(dim):
        v = float(f0[c])
        tol = 2.0 ** -22 * min(1 + np.exp(v), n) + (v + 8) * 2.0 ** -24
        for name, got, ref, k in (("y", y, y_ref, 1), ("final", fin, fin_ref, 1),
                                  ("df", g["df"], df, 2), ("dx", g["dx"], dx, 2),
                                  ("dinitial_state", g["dinitial_state"], dh0, 2)):
            _near(got[..., c], ref[..., c], (name, v), k * tol)


@pytest.mark.parametrize("n", [16, 17, 24, 31, 32, 33])
@pytest.mark.parametrize("batch,dim", [(26, 2560), (66, 1001), (1, 65535)])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_short_sequences_of_many_channels(n, batch, dim, dtype):
    """The lengths and channels where the forward's walk ends and the tiles begin, with pairs
    of channels and single ones to a thread."""
    _check(_inputs(batch, n, dim, dtype, n + dim))


@pytest.mark.parametrize("n", [12, 300])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_a_restart_ends_what_lies_behind_a_nan_gate(n, dtype):
    """A restart with a NaN gate after it in the same warp's steps, and a NaN gradient further
    on: nothing of it reaches the steps before the restart, nor the other way round."""
    d = _inputs(1, n, 70, dtype, n + 3)
    t = n // 2
    d["f"][0, t, 30], d["f"][0, t + 1, 30] = float("-inf"), float("nan")
    d["f"][0, t, 31], d["f"][0, t - 1, 31] = float("-inf"), float("nan")
    for c in (30, 31, 32):
        d["dy"][0, n - 1, c] = float("nan")
    dev, r = _dev(d), _n64(d)
    y, fin = binding.ssm_linrec_fwd(dev["f"], dev["x"], dev["z"], initial_state=dev["h0"])
    y_ref, fin_ref, _ = P.linrec_fwd(r["f"], r["x"], r["z"], r["h0"])
    _near(y, y_ref, "y", 1e-5)
    _near(fin, fin_ref, "final", 1e-5)
    refs = P.linrec_bwd(r["f"], r["x"], r["dy"], r["z"], r["h0"], r["dfin"])
    assert np.isfinite(refs[3][0, 30]) and np.isfinite(fin_ref[0, 31])
    assert np.isnan(refs[3][0, 31]) and np.isnan(refs[3][0, 32])
    g = binding.ssm_linrec_bwd(dev["f"], dev["x"], dev["dy"], dev["z"], initial_state=dev["h0"],
                               dfinal_state=dev["dfin"])
    for k, ref in zip(("df", "dx", "dz", "dinitial_state"), refs):
        _near(g[k], ref, k, 2e-5)
