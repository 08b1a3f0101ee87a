"""Shape's C struct belongs to whoever asked for it."""
import copy
import pickle

import video_dit_sequence_b200 as sp


def test_a_changed_struct_changes_no_later_call():
    shape = sp.Shape(1, 10, 4, 64, 2)
    mine = shape.c()
    mine.N, mine.H = 1000, 3
    assert [getattr(shape.c(), f) for f, _ in sp.sp_shape._fields_] == [1, 10, 4, 64, 2, 0.0]
    assert sp.check_shape(shape) == sp.SP_OK
    assert (shape._c.N, shape._c.H) == (10, 4)


def test_shapes_copy_and_travel():
    shape = sp.Shape(2, 37, 4, 128, 2, 0.25)
    shape.c(), shape.seq_sharded, shape.head_sharded, shape.lse_shape
    for other in (copy.copy(shape), copy.deepcopy(shape), pickle.loads(pickle.dumps(shape))):
        assert other == shape and hash(other) == hash(shape)
        assert bytes(other.c()) == bytes(shape.c())
