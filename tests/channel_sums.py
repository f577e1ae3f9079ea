"""How many additions in a row the weights' sums of the operators on channels
take, by the order that the kernels add in.  An oracle's bound for a sum is so
many roundings of its terms' magnitudes: counted generously, it also holds for
a result that has lost some of them."""


def _runs(offsets, shift):
    """{number: tokens} of the runs of at most 2^shift tokens, every sequence's
    from (its first token >> shift) + its number on."""
    runs = {}
    for s, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        for i, t in enumerate(range(lo, hi, 1 << shift)):
            runs[(lo >> shift) + s + i] = min(1 << shift, hi - t)
    return runs


def _most(runs, step, cost):
    """The most that the runs of one taker, every step-th, cost."""
    taken = {}
    for number, tokens in runs.items():
        taken.setdefault(number % step, []).append(tokens)
    return max((cost(t) for t in taken.values()), default=0)


def conv(offsets, T, channels, wide):
    """dweight and dbias of the convolution; `wide`: four channels a thread."""
    n = len(offsets) - 1
    lanes = -(-channels // (4 if wide else 1))
    waves = -(-lanes // 64)
    shift = 5
    while shift > 3 and ((T >> shift) + n) * waves < 4096:
        shift -= 1
    tx = 1
    while tx < lanes and tx < 64:
        tx *= 2
    side = 256 // tx
    parts = min(-(-((T >> shift) + n) // side), 128)
    # a thread goes on over its runs; then the block's threads, a quarter of
    # the parts, the four waves
    return _most(_runs(offsets, shift), parts * side, sum) + side + -(-parts // 4) + 3


def scan_tokens(offsets, T):
    """dA, dD and ddt_bias of the scan."""
    parts = min((T >> 7) + len(offsets) - 1, 512)
    # a segment's tokens (dA: times log2 e and ln 2, two roundings and two
    # constants; dD, ddt_bias: the four waves' sums), a workgroup's segments, a
    # quarter of the parts, the four waves
    return _most(_runs(offsets, 7), parts, lambda t: max(t) + len(t)) + 4 + -(-parts // 4) + 3


def scan_channels(channels, groups):
    """dB and dC of the scan: six folds of 64 lanes, at most four blocks in a
    workgroup, the workgroups."""
    blocks = -(-(channels // groups) // 64)
    return 6 + min(blocks, 4) + blocks
