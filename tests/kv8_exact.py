"""Inputs that the 8-bit cache holds without loss, and what attention over them
has to give, so that a page that is lost or counted twice shows.

Values are integers of -127..127 times a power of two, with a 127 in every
block: the block's scale is that power exactly and the codes are the integers.
Without a position rotation the queries are exact in half too, so of all that
the attention rounds only the weights, the scores' fp32 arithmetic and the
result remain."""
import numpy as np

PAGE = 16


def integers(rng, n, heads, d, step):
    """[n][heads][d] integers times step[page][head], a 127 in every block's first token."""
    x = rng.integers(-127, 128, (n, heads, d)).astype(np.float64)
    x[::PAGE, :, 0] = 127
    return x * np.repeat(step, PAGE, 0)[:n, :, None]


def steps(rng, n, heads, lo, hi):
    return 2.0 ** rng.integers(lo, hi + 1, (-(-n // PAGE), heads))


def marks(n, heads, d, first=0):
    """V of 127 in one dim of each page, 0 elsewhere: page p of head h marks dim (p + first + h) % d."""
    v = np.zeros((n, heads, d))
    page = np.arange(n) // PAGE
    for h in range(heads):
        v[np.arange(n), h, (page + first + h) % d] = 127
    return v


def mean_of_marks(pos, heads, d, first=0):
    """[len(pos)][heads][d]: the mean of marks() over positions 0..pos."""
    pos = np.asarray(pos, np.int64)
    full, rest = (pos + 1) // PAGE, (pos + 1) % PAGE
    out = np.zeros((len(pos), heads, d))
    for h in range(heads):
        for i in range(d):
            p0 = (i - first - h) % d  # the first page that marks i
            out[:, h, i] = PAGE * np.maximum(0, (full - p0 + d - 1) // d)
        out[np.arange(len(pos)), h, (full + first + h) % d] += rest
    return out * 127 / (pos + 1)[:, None, None]


def mean_bound(want):
    """Of a softmax scale of 0: the weights are 1 (in half exactly; the exponential of 0 or of next to 0 is within
    2^-23 of it), their sums whole numbers below 2^24 and so exact in fp32; 1 / sum and the product with it
    round by 2^-24 each, the result to bf16 by 2^-8."""
    return np.abs(want) * (2.0 ** -8 * (1 + 2.0 ** -20) + 2.0 ** -22)


def attention(q, k, v, pos0, scale):
    """q [n][nq][d] at pos0.., k, v [pos0 + n][heads][d] held without loss: (out, bound of a right result's error).

    With weights p_j = exp(x_j - max), their sum l, steps s_j and codes c_j (v_j = s_j c_j):
    - a weight p_j s_j is rounded to half: by 2^-11 of itself, and by 2^-25 of the largest p s where it falls
      below half's normal numbers;
    - a score x_j is off by e_j, which moves its weight by a factor exp(e_j) and the result by p_j e_j |v_j - out| / l:
      products are exact, an MMA's fp32 sum of d terms is cut at most 8 + 8 times (2^-23 each) and scaled in four
      roundings (2^-24): 2^-18 of the sum of its terms' magnitudes; the exponential's argument and
      value: 2^-21 (1 + |x_j| + |max|); query values below 2^-14 of their column's power of two lose 2^-25 of that power;
    - sums over up to n / 16 + 64 partial steps in fp32, cut (2^-23 of the sum of magnitudes each);
    - the result is rounded to bf16, 2^-8."""
    n, nq, d = q.shape
    group = nq // k.shape[1]
    out, tol = np.zeros((n, nq, d)), np.zeros((n, nq, d))
    unseen = np.arange(k.shape[0])[None] > pos0 + np.arange(n)[:, None]
    for h in range(nq):
        kh, vh = k[:, h // group], v[:, h // group]
        x = q[:, h] @ kh.T * scale
        x[unseen] = -np.inf
        top = x.max(1, keepdims=True)
        p = np.exp(x - top)
        l = p.sum(1, keepdims=True)
        out[:, h] = p @ vh / l
        step = np.repeat(np.abs(vh).reshape(len(vh), -1)[::PAGE].max(1) / 127, PAGE)[:len(vh)]
        mag = np.abs(q[:, h]) @ np.abs(kh).T * abs(scale)
        size = 2.0 ** np.floor(np.log2(np.abs(q[:, h]).max(1, keepdims=True)))
        e = 2.0 ** -18 * mag + 2.0 ** -21 * (1 + np.abs(np.where(unseen, 0, x)) + np.abs(top)) \
            + 2.0 ** -25 * size * np.abs(kh).sum(1)[None] * abs(scale)
        most = (p * step).max(1, keepdims=True)
        whole = p @ np.abs(vh)
        # sum_j p_j e_j |v_j - out| <= sum_j p_j e_j (|v_j| + |out|)
        err = (p * e) @ np.abs(vh) + (p * e).sum(1, keepdims=True) * np.abs(out[:, h])
        lost = 2.0 ** -25 * most * (np.where(unseen, 0, 1) @ (np.abs(vh) / step[:, None]))
        tol[:, h] = 2.0 ** -8 * np.abs(out[:, h]) + (2.0 ** -11 * whole + lost + 1.01 * err
                                                     + (k.shape[0] / 16 + 64) * 2.0 ** -23 * whole) / l
    return out, tol
