"""The tables of a generation step, request by request and token by token.  Test infrastructure only."""
import numpy as np


def tables(lengths, context, blocks, free_list, free_count, T, block, slots):
    """All books after the step and its tables, from copies of those before: a dict of int lists and arrays."""
    N = len(lengths)
    blocks, free_list = np.array(blocks), np.array(free_list)
    most = blocks.shape[1] * block if N else 0
    error = not 0 <= free_count <= slots
    count = 0 if error else int(free_count)
    after, good = [int(c) for c in context], []
    for n in range(N):
        ok = lengths[n] >= -1 and context[n] >= 0 and context[n] + max(lengths[n], 0) <= most
        good.append(ok)
        error |= not ok
    for n in range(N):
        if good[n] and lengths[n] == -1:
            for j in range(-(-int(context[n]) // block)):
                if count < slots:
                    free_list[count] = blocks[n][j]
                    count += 1
                else:
                    error = True
            after[n] = 0
    cu, positions, slot_out, slot_in = [0], [0] * T, [-1] * T, []
    waits = False
    for n in range(N):
        c, take = int(context[n]), int(lengths[n]) if good[n] and lengths[n] > 0 else 0
        held = -(-c // block)
        new = -(-(c + take) // block) - held if take else 0
        waits |= cu[-1] + take > T or new > count
        if waits:
            take = new = 0
        for j in range(held, held + new):
            count -= 1
            blocks[n][j] = free_list[count]
        slot_in.append(int(blocks[n][(c - 1) // block]) if good[n] and lengths[n] >= 0 and c > 0 else -1)
        for i in range(take):
            positions[cu[-1] + i] = c + i
            if i == take - 1 or (c + i + 1) % block == 0:
                slot_out[cu[-1] + i] = int(blocks[n][(c + i) // block])
        cu.append(cu[-1] + take)
        after[n] += take
    return dict(cu=cu, positions=positions, slot_in=slot_in, slot_out=slot_out, context=after, blocks=blocks, free_list=free_list,
                free_count=count, error=error)
