"""The numpy reference of the 4-bit row format against values worked out by hand (CPU)."""
import numpy as np

import quant_ref as R


def row(**groups):
    x = np.zeros(128)
    for name, vals in groups.items():
        g = int(name[1:])
        x[32 * g:32 * g + len(vals)] = vals
    return x


def test_levels_and_ties_by_hand():
    # amax 6: scale 1, so values are their own quotients; ties go to the even code
    x = row(g0=[6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -5, -0.25, 0.26, 0.74, 5.03125])
    codes, scales = R.hold(x)
    assert scales[0] == 1 and (scales[1:] == 0).all()
    back = R.values(codes, scales)
    assert list(back[:13]) == [6, 0, 1, 1, 2, 2, 4, 4, -4, 0, 0.5, 0.5, 6]
    assert (back[32:] == 0).all()


def test_byte_order_and_sign():
    codes, _ = R.hold(row(g0=[6, -6, 1.5, 0.5]))
    assert codes[0] == 0xF7 and codes[1] == 0x13


def test_scale_is_the_nearest_f16_and_is_capped():
    codes, scales = R.hold(row(g0=[7.0], g1=[2.0 ** 17], g2=[2.0 ** -26], g3=[0.01]))
    assert scales[0] == np.float16(7 / 6)
    assert scales[1] == np.float16(10912) and R.values(codes, scales)[32] == 65472
    assert scales[2] == 0 and R.values(codes, scales)[64] == 0
    assert scales[3] == np.float16(0.01 / 6)


def test_error_of_normal_rows():
    # a group's largest error is half the top step (scale) beside rounding of the scale
    x = R.round_bf16(np.random.default_rng(1).normal(size=(64, 128)))
    codes, scales = R.hold(x)
    err = np.abs(R.values(codes, scales) - x).reshape(64, 4, 32)
    s = scales.astype(np.float64)[..., None]
    assert (err <= s * (1 + 2.0 ** -7)).all()
    assert 0.05 < np.sqrt((err ** 2).mean()) < 0.15
    again, s2 = R.hold(R.round_bf16(R.values(codes, scales)))
    assert (np.abs(R.values(again, s2) - R.values(codes, scales)) <= 6 * 2.0 ** -7 * np.repeat(
        scales.astype(float), 32, -1)).all()


def test_decode_of_one_token_is_its_value_row():
    rng = np.random.default_rng(2)
    k, v = rng.normal(size=(2, 8, 2, 128)), rng.normal(size=(2, 8, 2, 128))
    q = rng.normal(size=(1, 4, 128))
    out, lse, _, _, _ = R.decode(q, k, v, [0, 1], np.array([1]), [1], "NHD", 0.1)
    np.testing.assert_allclose(out[0], np.repeat(v[1, 0], 2, 0))
    np.testing.assert_allclose(lse[0, :2], q[0, :2] @ k[1, 0, 0] * 0.1)


def test_rotation_keeps_norms_and_axes_move_only_their_pairs():
    x = np.random.default_rng(3).normal(size=(5, 2, 128))
    axis = [0] * 16 + [1] * 24 + [2] * 24
    pos = np.array([[0] * 5, [0] * 5, [3, 5, 7, 9, 11]])
    y = R.rotate(x, pos, axis, 1e4)
    np.testing.assert_array_equal(y[..., :40], x[..., :40])
    np.testing.assert_array_equal(y[..., 64:104], x[..., 64:104])
    np.testing.assert_allclose(y[..., :64] ** 2 + y[..., 64:] ** 2,
                               x[..., :64] ** 2 + x[..., 64:] ** 2)
    a = 11 * 10.0 ** -2.5  # pair 40 of the last token: 10000^(-80/128)
    np.testing.assert_allclose(y[4, 1, 40], x[4, 1, 40] * np.cos(a) - x[4, 1, 104] * np.sin(a))
