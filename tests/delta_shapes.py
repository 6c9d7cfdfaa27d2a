"""How the chunked calls of the gated delta rule cut a call's sizes (the rule of delta_shape in gla_delta_api.cpp, written
again), what their buffers hold, and sizes that take every kernel of it."""
import itertools

BF16, F32 = "bf16", "f32"
CHUNK, MARKS = 64, 4


def shape(B, H, T, dk, dv):
    """chunks N, segments P, a walk's waves NW, padded channels and values, marks."""
    N = -(-T // CHUNK)
    most = 1
    while most < N and (most + 1) ** 2 <= 9 * N:
        most += 1
    segments = lambda units: min(256 // units, most) if min(256 // units, most) >= 3 else 1  # noqa: E731
    wide = B * H * -(-dv // 128)
    NW = 4 if dv <= 64 or wide * segments(wide) <= 128 else 8
    L = -(-N // segments(B * H * -(-dv // (16 * NW))))
    return {"N": N, "P": -(-N // L), "NW": NW, "DKP": 32 if dk <= 32 else 64 if dk <= 64 else 128, "DVP": -(-dv // 16) * 16,
            "marks": -(-N // MARKS)}


def kind(B, H, T, dk, dv, dt):
    s = shape(B, H, T, dk, dv)
    return dt, s["DKP"], s["NW"], s["P"] > 1


KINDS = set(itertools.product((BF16, F32), (32, 64, 128), (4, 8), (False, True)))


def total(*regions):
    return sum(-(-n // 256) * 256 for n in regions)


def forward_bytes(B, H, Hk, T, dk, dv, dt):
    """The workspace of a forward: packed rows; the segments' states, in and out; inverses; transitions by rows; gates."""
    s, e = shape(B, H, T, dk, dv), 2 if dt == BF16 else 4
    heads, up = B * H, lambda d: -(-d // 8) * 8
    r = [heads * s["N"] * CHUNK * CHUNK * 4, heads * s["N"] * 5 * CHUNK * 4]
    r += [B * T * e * 2 * Hk * up(dk)] if dk % 8 else []
    r += [B * T * e * H * up(dv)] if dv % 8 else []
    if s["P"] > 1:
        r += [heads * s["P"] * s["DVP"] * s["DKP"] * 4] * 2 + [heads * s["P"] * s["DKP"] ** 2 * 4]
    return total(*r)


def saved_bytes(B, H, Hk, T, dk, dv, dt):
    """Gates, transposed inverses, transposed transitions, errors, o's rests, the states entering chunks, the marks."""
    s, e = shape(B, H, T, dk, dv), 2 if dt == BF16 else 4
    heads = B * H
    chunks, row = heads * s["N"], CHUNK * s["DVP"]
    r = [chunks * 5 * CHUNK * 4, chunks * CHUNK * CHUNK * 4, chunks * row * 4, chunks * s["DVP"] * s["DKP"] * e,
         heads * (s["marks"] + 1) * s["DVP"] * s["DKP"] * 4]
    r += [heads * s["P"] * s["DKP"] ** 2 * 4] if s["P"] > 1 else []
    r += [chunks * row * 2] if dt == BF16 else []
    return total(*r)


# B, H, Hk, T, dk, dv, dtype, lengths or None: 128 columns a workgroup (8 waves) and 64, whole and in segments of one and of
# several chunks, with 32, 64 and 128 channels, in both types; keys shared, odd widths, a last tile of few columns
CASES = [(b, h, hk, t, dk, dv, dt, lens) for dt in (BF16, F32) for b, h, hk, t, dk, dv, lens in (
    (1, 17, 17, 700, 128, 128, None), (1, 9, 3, 700, 100, 200, (650,)), (2, 9, 9, 640, 64, 80, (640, 391)),
    (1, 17, 17, 450, 24, 100, None), (1, 86, 86, 70, 128, 128, None), (2, 65, 65, 66, 128, 128, None), (2, 35, 35, 130, 72, 130, (130, 3)),
    (1, 90, 45, 130, 64, 72, None), (1, 130, 65, 130, 64, 72, None), (1, 140, 70, 70, 32, 100, None), (1, 2, 1, 300, 128, 64, None), (1, 2, 2, 300, 40, 48, None),
    (1, 3, 1, 500, 16, 300, (444,)), (1, 3, 3, 64, 128, 96, None), (2, 2, 2, 60, 64, 200, (60, 31)), (1, 2, 2, 33, 30, 64, None))]
