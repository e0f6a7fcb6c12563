"""Which of the dense attention kernels works on a batch: what a call left in
its workspace, and the device's rule restated."""
import torch

PAIR, QUAD, SINGLE = 0, 1, 2


def kinds(workspace):
    """The kinds of the groups of CTAs that left cut row tiles in a call's
    workspace (filled with 0xFF before): behind the partials and their (max,
    sum) lie the cut row tiles' descriptors, (first row, rows, further parts,
    kind) each."""
    sms = torch.cuda.get_device_properties(workspace.device).multi_processor_count
    rows = 2 * (sms // 2) * 128
    desc = workspace[rows * (512 * 4 + 8):][:16 * sms].view(torch.int32).view(-1, 4).cpu()
    return set(desc[desc[:, 2] > 0, 3].tolist())


def takes_quads(lens, q_lens, H, quads=36):
    """Whether clusters of four work on this batch as one (not as two pairs)."""
    if sum(q_lens) * H < 256 * len(lens):
        return False
    cost = []
    for rows, tile, step in ((128, 71, 44), (256, 123, 27)):
        tokens = rows // H
        c = 0
        for n, m in zip(lens, q_lens):
            for t in range(0, m, tokens):
                seen = n if n < m else n - m + min(m, t + tokens)
                c += tile + step * max(1, -(-seen // 128))
        cost.append(c)
    return 2 * cost[1] + 240 * quads < cost[0]
