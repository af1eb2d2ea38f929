"""The handshake of the attention kernel for many rows (turns: units of 128 rows, two softmax warpgroups
taking turns with the blocks), explored over every order in which its roles can run.

Each role is the list of its waits, arrivals and products for given units; a state is how far every role and the
tensor pipe have come and how many phases each barrier has completed.  Barriers are waited for by the parity of a phase,
as mbarrier.try_wait.parity does: true while the present phase's parity differs from the one asked for."""
import pytest


def roles(units, both_see=True):
    """The roles' programs for units of the given numbers of blocks, and the barriers' arrival counts.  One warp stands
    for a role's warps.  K and V are always there (they wait for the products alone).  both_see: P's barrier also
    takes an arrival of the warpgroup whose turn the block is not, once it has seen the block's S."""
    owner, first, last = [], [], []
    for blocks in units:
        for x in range(blocks):
            owner.append(len(owner) & 1)
            first.append(x == 0)
            last.append(x == blocks - 1)
    n = len(owner)

    def half(i):                                  # the barrier of block i and the parity of its phase
        return i & 1, i >> 1 & 1

    issue, units_o = [], 0

    def product_o(i):
        nonlocal units_o
        b, p = half(i)
        issue.append(("wait", f"vp{b}", p))
        if first[i]:
            if units_o:
                issue.append(("wait", "o_free", units_o - 1 & 1))
            units_o += 1
        issue.append(("product",))
        issue.append(("commit", f"o{b}"))

    for i in range(n + 1):
        if i and last[i - 1]:
            product_o(i - 1)
        if i == n:
            break
        issue += [("product",), ("commit", f"s{i & 1}")]
        if i and not last[i - 1]:
            product_o(i - 1)
    issue += [("commit", f"s{n & 1}"), ("commit", f"s{n + 1 & 1}")]

    softmax = []
    for wg in range(2):
        prog, unit = [], 0
        for i in range(n):
            b, p = half(i)
            before, bp = half(i - 1)
            prog.append(("wait", f"s{b}", p))
            if owner[i] != wg and both_see:
                prog.append(("arrive", f"vp{b}"))
            if owner[i] == wg:
                if not first[i]:
                    prog.append(("wait", f"m{before}", bp))
                prog.append(("arrive", f"m{b}"))
                if not first[i]:
                    prog.append(("maybe", f"o{before}", bp))          # only where a reference is raised
                prog.append(("arrive", f"vp{b}"))
            if last[i]:
                if owner[i] != wg:
                    prog.append(("wait", f"m{b}", p))
                prog += [("arrive", "l"), ("wait", "l", unit & 1), ("wait", f"o{b}", p), ("arrive", "o_free")]
                unit += 1
        prog.append(("wait", f"s{n & 1}", n >> 1 & 1))
        softmax.append(prog)
    counts = {"l": 2, "o_free": 2, "vp0": 1 + both_see, "vp1": 1 + both_see}
    return [issue] + softmax, counts


def explore(programs, counts, expire=False, drain=None):
    """Every reachable end: 'done', 'stuck' (a role waits for ever) and, where waits may expire (which sets the abort
    flag and sends the role to its end), 'early' if tensor memory is freed while a product is under way.  drain: what the
    issuing role's last wait does once the flag is set: 'leaves' or 'waits'."""
    names = sorted({op[1] for p in programs for op in p if len(op) > 1}) + ["drain"]
    at = {b: i for i, b in enumerate(names)}
    need = [counts.get(b, 1) for b in names]

    def arrive(bars, b):
        bars = list(bars)
        phases, have = bars[at[b]]
        have += 1
        bars[at[b]] = (phases + 1, 0) if have == need[at[b]] else (phases, have)
        return tuple(bars)

    # a role's place: index of its next op; len + 1: at its end (after the issuing role's drain)
    start = (tuple(0 for _ in programs), (), tuple((0, 0) for _ in names), False)
    seen, todo, ends = {start}, [start], set()
    while todo:
        pcs, pipe, bars, flag = todo.pop()
        out = []
        if pipe:                                  # the tensor pipe: products and commits in order
            out.append((pcs, pipe[1:], arrive(bars, pipe[0]) if pipe[0] else bars, flag))
        for r, prog in enumerate(programs):
            pc = pcs[r]

            def to(x, pipe=pipe, bars=bars, flag=flag):
                out.append((pcs[:r] + (x,) + pcs[r + 1:], pipe, bars, flag))

            if pc > len(prog):
                continue
            if pc == len(prog):
                if r or drain is None:
                    to(pc + 1)
                elif bars[at["drain"]][0] or (drain == "leaves" and flag):
                    to(pc + 1)
                continue

            def end():                            # the issuing role's drain is committed as it gets there
                return pipe + ("drain",) if r == 0 and drain is not None else pipe

            op = prog[pc]
            over = pc + 1 == len(prog)
            if op[0] in ("wait", "maybe"):
                if (bars[at[op[1]]][0] & 1) != op[2] or op[0] == "maybe":
                    to(pc + 1, pipe=end() if over else pipe)
                if expire and op[0] == "wait" and (bars[at[op[1]]][0] & 1) == op[2]:
                    to(len(prog), pipe=end(), flag=True)
            elif op[0] == "arrive":
                to(pc + 1, bars=arrive(bars, op[1]))
            else:
                x = "" if op[0] == "product" else op[1]
                more = pipe + (x,)
                to(pc + 1, pipe=more + ("drain",) if over and r == 0 and drain is not None else more)
        if all(pc == len(p) + 1 for pc, p in zip(pcs, programs)):
            if drain is not None and "" in pipe:
                ends.add("early")
            elif not pipe:
                ends.add("done")
        elif not out:
            ends.add("stuck")
        for s in out:
            if s not in seen:
                seen.add(s)
                todo.append(s)
    return ends


UNITS = [[1], [2], [3], [4], [7], [1, 1, 1, 1], [3, 1, 2], [1, 4], [2, 3, 2], [2, 1, 2, 1, 3]]


@pytest.mark.parametrize("units", UNITS, ids=str)
def test_no_order_of_the_roles_gets_stuck(units):
    assert explore(*roles(units)) == {"done"}


def test_a_block_that_one_warpgroup_has_not_seen_is_what_would_get_stuck():
    """Were the products to wait for the block's own warpgroup alone, a late warp of the other one could find S's barrier
    two phases on, which by its parity looks like none."""
    assert "stuck" in explore(*roles([4], both_see=False))


def test_tensor_memory_outlives_the_products():
    """A role gives up at any wait: the issuing role's last wait is for its own products, whether or not the flag is
    set.  (Left at the flag, memory is freed under them: the check tells the two apart.)"""
    programs, counts = roles([2, 1])
    assert "early" in explore(programs, counts, expire=True, drain="leaves")
    for units in UNITS:
        assert explore(*roles(units), expire=True, drain="waits") == {"done"}
