"""m2_state_reorder: the paged states after a beam selection, against the rule
written out row by row.  Copies are exact; every slot that is not a copy's
target keeps its bytes."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

m2 = pytest.importorskip("mamba2_ssm_mixer_gb300")

CONV, SSM = (6144, 3), (64, 64, 128)


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _rule(slots, parents):
    """New slots and the copies (to, from) of valid requests."""
    new, moves = np.full_like(slots, -1), []
    for i, (row, par) in enumerate(zip(slots.tolist(), parents.tolist())):
        spare = [s for j, s in enumerate(row) if s >= 0 and j not in par]
        seen = set()
        for j, p in enumerate(par):
            if p >= 0 and p not in seen:
                new[i, j] = row[p]
                seen.add(p)
            elif p >= 0:
                new[i, j] = spare.pop(0)
                moves.append((int(new[i, j]), row[p]))
        for j, p in enumerate(par):
            if p < 0 and spare:
                new[i, j] = spare.pop(0)
    return new, moves


def _pools(layers, n_slots, dtype, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    conv = [torch.randn((n_slots, *CONV), generator=g, device="cuda").to(torch.bfloat16) for _ in range(layers)]
    ssm = [torch.randn((n_slots, *SSM), generator=g, device="cuda").to(dtype) for _ in range(layers)]
    return conv, ssm


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def _run(slots, parents, conv, ssm, **kw):
    keep = [[t.clone() for t in p] for p in (conv, ssm)]
    new = m2.m2_state_reorder(conv, ssm, _dev(slots), _dev(parents), **kw)
    torch.cuda.synchronize()
    return new.cpu().numpy(), keep


def _expect(slots, parents, conv, ssm, new, keep):
    want, moves = _rule(slots, parents)
    assert np.array_equal(new, want)
    for now, was in ((conv, keep[0]), (ssm, keep[1])):
        for a, b in zip(now, was):
            if moves:
                to, of = (torch.tensor(v, device="cuda") for v in zip(*moves))
                b[to] = b[of]
            assert torch.equal(a, b)


@pytest.mark.parametrize("batch,beams,layers,n_slots,dtype", [
    (1, 1, 1, 1, torch.float32), (1, 4, 1, 4, torch.float32), (3, 5, 2, 20, torch.bfloat16),
    (1, 32, 1, 40, torch.bfloat16), (7, 3, 3, 64, torch.float32), (9, 8, 1, 72, torch.bfloat16)])
def test_follows_the_rule(batch, beams, layers, n_slots, dtype):
    rng = np.random.default_rng(batch * 100 + beams)
    conv, ssm = _pools(layers, n_slots, dtype)
    slots = rng.permutation(n_slots)[:batch * beams].reshape(batch, beams)
    for _ in range(3):
        parents = rng.integers(0, beams, (batch, beams))
        new, keep = _run(slots, parents, conv, ssm)
        _expect(slots, parents, conv, ssm, new, keep)
        assert np.array_equal(np.sort(new, 1), np.sort(slots, 1))
        slots = new
    m2.check_standalone()


@pytest.mark.parametrize("parents", [[0, 1, 2, 3], [3, 2, 1, 0], [2, 2, 2, 2], [1, 1, -1, 0], [-1, -1, -1, -1],
                                     [3, -1, 3, 3]])
def test_one_request(parents):
    conv, ssm = _pools(1, 6, torch.float32)
    slots, parents = np.array([[5, 0, 3, 2]]), np.array([parents])
    new, keep = _run(slots, parents, conv, ssm)
    _expect(slots, parents, conv, ssm, new, keep)
    m2.check_standalone()


def test_rows_without_a_slot():
    """A request with fewer slots than rows: rows with no slot can be nobody's
    parent; as many rows live as there are slots."""
    conv, ssm = _pools(1, 8, torch.float32)
    slots = np.array([[4, -1, 2, -1], [-1, -1, -1, -1], [7, 6, 5, -1]])
    parents = np.array([[2, 2, -1, -1], [-1, -1, -1, -1], [0, 0, 1, -1]])
    new, keep = _run(slots, parents, conv, ssm)
    _expect(slots, parents, conv, ssm, new, keep)
    assert new.tolist() == [[2, 4, -1, -1], [-1, -1, -1, -1], [7, 5, 6, -1]]
    m2.check_standalone()


@pytest.mark.parametrize("bad", ["slot high", "slot low", "slot twice", "slot of another request", "parent high",
                                 "parent low", "parent without slot", "more rows than slots"])
def test_a_wrong_request_is_left_alone_and_reported(bad):
    conv, ssm = _pools(2, 16, torch.bfloat16)
    slots = np.array([[0, 1, 2], [3, 4, 5], [6, 7, 8]])
    parents = np.array([[1, 1, 0], [2, 2, 2], [0, 0, 1]])
    if bad == "slot high":
        slots[1, 0] = 16
    elif bad == "slot low":
        slots[1, 0] = -2
    elif bad == "slot twice":
        slots[1, 0] = 5
    elif bad == "slot of another request":
        slots[1, 0] = 2
    elif bad == "parent high":
        parents[1, 1] = 3
    elif bad == "parent low":
        parents[1, 1] = -2
    elif bad == "parent without slot":
        slots[1, 2] = -1
    else:
        slots[1, 0] = -1
    new, keep = _run(slots, parents, conv, ssm)
    assert np.array_equal(new[1], slots[1])
    good = [0, 2]
    _expect(slots[good], parents[good], conv, ssm, new[good], keep)
    with pytest.raises(m2.M2Error) as e:
        m2.check_standalone()
    assert e.value.status == m2.M2_EINVAL
    m2.check_standalone()


def test_no_requests():
    conv, ssm = _pools(1, 2, torch.float32)
    none = torch.empty((0, 4), dtype=torch.int32, device="cuda")
    assert m2.m2_state_reorder(conv, ssm, none, none).shape == (0, 4)


def test_the_most_rows():
    """4096 rows, every slot named: the plan alone (each beam goes on as
    itself, permuted), and one copy."""
    conv, ssm = _pools(1, 64, torch.bfloat16)
    rng = np.random.default_rng(1)
    slots = np.full((128, 32), -1)
    slots[5], slots[77] = rng.permutation(64).reshape(2, 32)
    parents = np.full((128, 32), -1)
    parents[5], parents[77] = rng.permutation(32), rng.permutation(32)
    parents[77][0] = parents[77][1]
    new, keep = _run(slots, parents, conv, ssm)
    _expect(slots, parents, conv, ssm, new, keep)
    m2.check_standalone()


def test_captured_and_on_two_streams():
    conv, ssm = _pools(2, 32, torch.float32)
    rng = np.random.default_rng(3)
    slots = rng.permutation(32).reshape(4, 8)
    parents = rng.integers(0, 8, (4, 8))
    keep = [[t.clone() for t in p] for p in (conv, ssm)]
    sd, pd, out = _dev(slots), _dev(parents), torch.empty((4, 8), dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m2.m2_state_reorder(conv, ssm, sd, pd, out=out)
    parents = rng.integers(0, 8, (4, 8))
    pd.copy_(_dev(parents))
    g.replay()
    g.replay()                                  # the same copies again change nothing
    torch.cuda.synchronize()
    _expect(slots, parents, conv, ssm, out.cpu().numpy(), keep)
    # two halves of the requests on two streams at once
    slots = out.cpu().numpy()
    parents = rng.integers(0, 8, (4, 8))
    keep = [[t.clone() for t in p] for p in (conv, ssm)]
    halves = [(_dev(slots[h]), _dev(parents[h]), torch.cuda.Stream()) for h in (slice(0, 2), slice(2, 4))]
    torch.cuda.synchronize()
    new = [m2.m2_state_reorder(conv, ssm, s, p, stream=st) for s, p, st in halves]
    torch.cuda.synchronize()
    _expect(slots, parents, conv, ssm, torch.cat(new).cpu().numpy(), keep)
    m2.check_standalone()


def test_reorder_then_decode_sees_the_copies():
    """A pre-quantised decode directly behind the reorder (its state loads
    start early) equals one after a synchronize."""
    import synth
    from helpers import device_weights
    blk = m2.Mamba2Mixer(device_weights(synth.make_weights(0)))
    slots = np.arange(8).reshape(1, 8)
    parents = np.array([[3, 3, 3, 1, 1, 0, 7, 7]])
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    q = torch.randint(0, 100, (8, 2688), generator=g, device="cuda", dtype=torch.uint8)
    outs = []
    for sync in (True, False):
        conv, ssm = _pools(1, 8, torch.float32, 9)
        for _ in range(3):
            new = m2.m2_state_reorder(conv, ssm, _dev(slots), _dev(parents))
            if sync:
                torch.cuda.synchronize()
            out = blk.decode(q, conv[0], ssm[0], new.view(-1))
            if sync:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        outs.append((out, conv[0], ssm[0]))
    blk.check()
    m2.check_standalone()
    assert all(torch.equal(a, b) for a, b in zip(*outs))
