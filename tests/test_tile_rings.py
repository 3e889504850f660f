"""The rings between the tile GEMM's copies, decoder groups and matrix instructions: a model of their
waits, searched over every order in which copies can land and roles can run.

A wait on a slot's barrier is by parity, so it also passes when the slot is a whole phase behind.  The
model counts what a slot has really completed and reports a wait that passes without its own step."""
import ctypes

import pytest

import fp8_weight_only_w4a16_b200 as sk

KERNELS = [(fmt, w) for fmt in (sk.FMT_NVFP4, sk.FMT_FP8) for w in (16, 32, 64, 128, 192)]


def rings(fmt, width):
    out = (ctypes.c_int * 4)()
    assert sk.library().skinny_debug_tile_rings(fmt, width, out) == sk.OK
    return tuple(out)


def passes_early(weights, tokens, groups, waits_for_slot, steps=13):
    """(what, step) of a wait that can pass before its own step has completed, or None.

    Step s belongs to group s % groups, its weights lie in slot s % weights, its tokens' slot s % tokens
    is free again when the matrix instructions of step s are done, which run in order."""

    def done(count, slot, slots):             # completed phases of a slot when `count` steps are done, in order
        return (count - 1 - slot) // slots + 1 if count > slot else 0

    def wait(phases, wanted):                 # (passes, rightly): the barrier knows the parity only
        return phases % 2 == wanted % 2, phases >= wanted

    # own steps finished by each group, and whether its next one is decoded; matrix instructions done;
    # copies issued; which of them have landed
    start = ((0,) * groups, (False,) * groups, 0, 0, 0)
    seen, todo = {start}, [start]
    while todo:
        own, decoded, mma, issued, landed = state = todo.pop()
        following = []
        freed = issued - weights
        if issued < steps and (freed < 0 or own[freed % groups] > freed // groups):
            following.append((own, decoded, mma, issued + 1, landed))
        following += [(own, decoded, mma, issued, landed | 1 << s) for s in range(issued) if not landed >> s & 1]
        if mma < steps and own[mma % groups] > mma // groups:
            following.append((own, decoded, mma + 1, issued, landed))
        for g in range(groups):
            s = own[g] * groups + g
            if s >= steps:
                continue
            if not decoded[g]:
                if waits_for_slot and s >= tokens:
                    ok, right = wait(done(mma, s % tokens, tokens), (s - tokens) // tokens + 1)
                    if ok and not right:
                        return "token slot", s
                    if not ok:
                        continue
                phases = sum(landed >> t & 1 for t in range(s % weights, steps, weights))
                ok, right = wait(phases, s // weights + 1)
                if ok and not right:
                    return "weights", s
                if ok:
                    following.append((own, decoded[:g] + (True,) + decoded[g + 1:], mma, issued, landed))
            else:
                last = s - groups             # the decoded stage is free when its matrix instructions are done
                if last >= 0:
                    ok, right = wait(done(mma, last % tokens, tokens), last // tokens + 1)
                    if ok and not right:
                        return "decoded stage", s
                    if not ok:
                        continue
                following.append((own[:g] + (own[g] + 1,) + own[g + 1:], decoded[:g] + (False,) + decoded[g + 1:], mma,
                                  issued, landed))
        assert following or mma == steps, "a state that no role can leave"
        for n in following:
            if n not in seen:
                seen.add(n)
                todo.append(n)
    return None


def test_the_model_finds_rings_that_are_too_short():
    assert passes_early(3, 3, 2, False) is not None         # the slot's last copy was another group's
    assert passes_early(4, 11, 3, False) is not None
    for weights in (2, 4, 5, 6):
        assert passes_early(weights, 3, 2, False) is None


@pytest.mark.parametrize("fmt,width", KERNELS)
def test_no_wait_of_the_decoders_passes_early(fmt, width):
    weights, tokens, groups, waits = rings(fmt, width)
    assert groups == 2
    assert passes_early(weights, tokens, groups, bool(waits)) is None


def test_refusals():
    out = (ctypes.c_int * 4)()
    call = sk.library().skinny_debug_tile_rings
    assert call(-1, 256, out) == sk.OK and out[2] == 0
    for fmt, width in ((0, 256), (1, 48), (-1, 192), (2, 16), (-2, 16)):
        assert call(fmt, width, out) == sk.ERR_INVALID_ARG
    assert call(0, 16, None) == sk.ERR_INVALID_ARG
