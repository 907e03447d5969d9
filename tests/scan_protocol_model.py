"""A randomised model of how the two halves of a delta-rule scan CTA hand each other their lane maxima.

Test infrastructure: ``tests/test_scan_protocol.py`` runs it on the CPU.  It mirrors the loop over the chunks of
``scan_head`` in ``rma_gdn_prefill.cu``: one warp of each half (they own the same value columns) and the warp that issues
the products, with the barriers between them.  Per chunk a half takes the other's maxima, waits for W, gives X, waits
for U, gives the scaled U, waits for the state's increment, offers its new maxima and gives the state.

Waits on mbarriers are bounded: at random one runs out, the CTA's abort flag is up from then on, every such wait returns
at once, the halves go on through their barriers on values that nobody uses, and the issuing warp leaves.  ``hand_over``
selects what the maxima go by: the bounded wait for the other half's ``"state"``, as in the kernel, or a ``"named"`` barrier
of both warps (an arrival by the one, an arrival and an unbounded wait by the other).

Checked: every role comes to its end (Deadlock otherwise); without a timeout a half always takes the maxima of its own
chunk, and no barrier is two phases ahead of a wait on it.
"""
import random


class Deadlock(Exception):
    pass


class Barrier:
    def __init__(self, count):
        self.count, self.pending, self.done = count, count, 0

    def arrive(self):
        self.pending -= 1
        if self.pending == 0:
            self.pending, self.done = self.count, self.done + 1


def run(chunks, seed, timeout_rate=0.0, hand_over="state"):
    rng = random.Random(seed)
    abort = [False]
    S, X, U, UDone = ([Barrier(1), Barrier(1)] for _ in range(4))
    WDone, DDone = Barrier(1), Barrier(1)
    offered = [Barrier(2), Barrier(2)]   # the named barriers
    both = Barrier(2)
    slot = [None, None]

    def bounded(bar, phase):
        """A bounded wait: True when the phase is complete, False once the CTA is abandoned."""
        while bar.done <= phase:
            if abort[0]:
                return False
            if rng.random() < timeout_rate:
                abort[0] = True
                return False
            yield
        assert abort[0] or bar.done <= phase + 1, "two phases ahead of a wait"
        return True

    def offer(g, what):
        slot[g] = what
        if hand_over == "named":
            offered[g].arrive()

    def meet():
        phase = both.done
        both.arrive()
        while both.done == phase:
            yield

    def take(g, what):
        bar = offered[1 - g]
        if hand_over == "state":
            yield from (bounded(S[1 - g], what - 1) if what else meet())
        else:
            phase = bar.done
            bar.arrive()
            while bar.done == phase:
                yield
        assert abort[0] or slot[1 - g] == what, "another chunk's maxima"

    def half(g):
        offer(g, 0)
        yield from take(g, 0)
        yield from meet()
        for c in range(-1, chunks):
            if c >= 0:
                yield from take(g, c + 1)
                yield from bounded(WDone, c)
                X[g].arrive()
                yield from bounded(UDone[g], c)
                U[g].arrive()
                yield from bounded(DDone, c)
            if c + 1 < chunks:
                offer(g, c + 2)
                yield
                S[g].arrive()
            yield

    def products():
        for c in range(chunks):
            for bar, then in ((S[0], None), (S[1], WDone), (X[0], UDone[0]), (X[1], UDone[1]), (U[0], None), (U[1], DDone)):
                if not (yield from bounded(bar, c)):
                    return
                yield
                if then is not None:
                    then.arrive()

    roles = [half(0), half(1), products()]
    idle = 0
    while roles:
        role = rng.choice(roles)
        before = (len(roles), abort[0], [b.done for b in (*S, *X, *U, *UDone, WDone, DDone, *offered, both)], slot[:])
        for _ in range(rng.choice((1, 1, 2, 7))):   # a role may run ahead of the others
            try:
                next(role)
            except StopIteration:
                roles.remove(role)
                break
        after = (len(roles), abort[0], [b.done for b in (*S, *X, *U, *UDone, WDone, DDone, *offered, both)], slot[:])
        idle = 0 if before != after else idle + 1
        if idle > 2000:
            raise Deadlock(f"{len(roles)} roles wait for good")
    return abort[0]
