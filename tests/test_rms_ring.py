"""Host-side: the sizes of tests/test_gpu_rms_ring.py go round the norm's rings in shared memory, and fill stages with more rows
than the warps take in one turn, in each form of the kernels.  The rules of rms_elements.cu and rms_norm.cu restated, for 152
SMs."""
from test_gpu_rms_ring import SIZES

SMS, WARPS, MOST_STAGES = 152, 8, 8


def _stream_rows(M, at_once, tensors, row_bytes, ctas):
    if at_once == 1:
        return 1
    times = min(24 * 1024 // (at_once * tensors * row_bytes), M // (2 * at_once * ctas))
    return at_once * min(max(times, 1), 16)


def ring(M, C, size, backward, residual, ctas=None):
    """(form, rows that the warps take in a turn, rows of a stage, stages, the most groups of rows that a CTA takes); None:
    no ring."""
    vec = 16 // size
    if C % vec:  # by elements
        if C > 8192:
            return None
        at_once = WARPS if C <= 1024 else 1
        ctas = 2 * SMS
        rows = _stream_rows(M, at_once, 3 if backward else 2, C * size, ctas)
        tensors = (2 if backward else 1) + residual
        stage = tensors * ((rows * C * size + 14 + 15) // 16 * 16)
        stages = 112 * 1024 // stage or 225 * 1024 // stage
        form = "elements, %d warps" % (1 if at_once > 1 else WARPS)
    else:
        granules = C // vec
        if not backward or granules > 1024:
            return None
        lanes = 8 if granules <= 8 else 16 if granules <= 16 else 32 if granules <= 128 else 256
        items = 1 if granules <= lanes else 2 if granules <= 2 * lanes else 4
        per_sm = 1 if items == 4 else 2
        at_once, ctas = 32 * WARPS // lanes, per_sm * SMS
        rows = _stream_rows(M, at_once, 3, C * size, ctas)
        stages = ((113 if per_sm == 2 else 226) * 1024 - 1024) // (3 * C * size * rows)
        form = "%d lanes" % lanes
    groups = -(-M // rows)
    return form, at_once, rows, min(stages, MOST_STAGES), -(-groups // ctas)


def test_the_sizes_go_round_the_rings():
    for size in (2, 4):
        for backward in (False, True):
            for residual in (False, True):
                wrapped, deep = set(), set()
                for M, C in SIZES:
                    r = ring(M, C, size, backward, residual)
                    if r is None:
                        continue
                    form, at_once, rows, stages, turns = r
                    if turns > stages:
                        wrapped.add(form)
                        if rows > at_once:
                            deep.add(form)
                forms = {"elements, 1 warps", "elements, 8 warps"} | ({"8 lanes", "16 lanes", "32 lanes", "256 lanes"} if backward else set())
                assert wrapped == forms, (size, backward, residual, forms - wrapped)
                assert deep >= {"elements, 1 warps"} | ({"8 lanes", "16 lanes"} if backward else set()), (size, backward, residual, deep)
