"""The functional forms keep a bounded number of plans, the ones used last (host-side)."""
import weakref

from cnn_convolution_implicit_gb300 import binding, operators


class Plan:
    pass


def test_the_plan_used_longest_ago_makes_room():
    cache = binding.PlanCache(limit=3)
    gone = {}
    for k in "abc":
        plan = Plan()
        gone[k] = weakref.ref(plan)
        assert cache.get(k) is None and cache.put(k, plan) is plan
    del plan
    assert cache.get("a") is gone["a"]()          # "b" is now the one used longest ago
    held = cache.get("b"), cache.get("a"), cache.get("c")
    cache.put("d", Plan())
    assert cache.get("b") is None and len(cache) == 3
    assert gone["b"]() is held[0]                 # a call under way still holds it
    del held
    assert gone["b"]() is None and gone["a"]() is not None
    cache.clear()
    assert len(cache) == 0 and gone["a"]() is None


def test_every_functional_form_is_bounded():
    caches = binding._plan_cache, operators._norm_plans, operators._int8_plans
    assert all(isinstance(c, binding.PlanCache) for c in caches)
    assert sum(c.limit for c in caches) < 1024    # status words of the device
