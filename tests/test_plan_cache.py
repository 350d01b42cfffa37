"""The functional forms keep a bounded number of plans, the ones used last (host-side)."""
import weakref

from cnn_convolution_implicit_gb300 import binding, operators


class Plan:
    pass


def test_a_plan_that_nobody_took_lately_makes_room():
    cache = binding.PlanCache(limit=3)
    gone = {}
    for k in "abc":
        plan = Plan()
        gone[k] = weakref.ref(plan)
        assert cache.get(k) is None and cache.put(k, plan) is plan
    del plan
    held = cache.get("a")
    held.used = True                              # as a call does
    cache.put("d", Plan())                        # "a" loses its mark and its place, "b" goes
    assert set(cache) == {"a", "c", "d"} and gone["b"]() is None
    cache.put("e", Plan())
    assert set(cache) == {"a", "d", "e"} and gone["c"]() is None
    for k in "fghij":
        cache.put(k, Plan())
        assert len(cache) == 3 and cache.get(k) is not None
    assert cache.get("a") is None and gone["a"]() is held   # a call under way still holds it
    del held
    assert gone["a"]() is None
    cache.clear()
    assert len(cache) == 0


def test_a_plan_in_use_stays():
    cache = binding.PlanCache(limit=8)
    hot = cache.put("hot", Plan())
    for k in range(1000):
        assert cache.get("hot") is hot
        hot.used = True
        cache.put(k, Plan())
    assert len(cache) == 8


def test_every_functional_form_is_bounded():
    caches = binding._plan_cache, operators._norm_plans, operators._int8_plans
    assert all(isinstance(c, binding.PlanCache) for c in caches)
    assert sum(c.limit for c in caches) < 1024    # status words of the device
