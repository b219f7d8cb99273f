"""The few-token layer's K split, restated: how many warps a team has, from the sizes of a call."""

WARPS = 16  # of a block, one block an SM


def choose(units, sms, nch):
    """The power of two S that leaves the busiest warp the fewest chunks, a join counted as one."""
    best = None
    for S in (1, 2, 4, 8, 16):
        if S > nch:
            break
        cost = -(-units // (sms * WARPS // S)) * (-(-nch // S) + (S > 1))
        if best is None or cost < best[0]:
            best = (cost, S)
    return best[1]


def of_call(counts, H, I, sms):
    """S of gate_up and of down for the tokens that each expert got."""
    slots = sum(-(-int(c) // 8) for c in counts)
    return (choose(slots * (I // 32), sms, H // 128), choose(slots * (H // 64), sms, -(-I // 128)))
